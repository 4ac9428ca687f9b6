// Whether an output shares bytes with what a call reads (host): outputs are written while other
// workgroups still read, so such a call would be a race.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "common.h"

namespace exmoe {

// groups of rows of `bytes` bytes, ld bytes apart, the groups stride bytes apart
struct MemRows {
  const char* name;
  const void* p;   // null: nothing
  size_t groups, stride, rows, ld, bytes;
};
inline MemRows mem_flat(const char* name, const void* p, size_t bytes) { return {name, p, 1, 0, 1, 0, bytes}; }
inline MemRows mem_matrix(const char* name, const void* p, size_t rows, size_t ld, size_t cols, size_t size) {
  return {name, p, 1, 0, rows, ld * size, cols * size};
}
inline MemRows mem_matrices(const char* name, const void* p, size_t groups, size_t stride, size_t rows, size_t ld,
                            size_t cols, size_t size) {
  if (groups == 1 || stride == rows * ld) return mem_matrix(name, p, groups * rows, ld, cols, size);
  return {name, p, groups, stride * size, rows, ld * size, cols * size};
}

typedef unsigned __int128 wide_t;   // (ends of strided operands may lie past 64 bits before they are refused)

// na rows of ca bytes from a on, lda apart, against nb rows of cb bytes from b on.
inline bool rows_overlap(wide_t a, size_t na, size_t lda, size_t ca, wide_t b, size_t nb, size_t ldb, size_t cb) {
  if (a + (wide_t)(na - 1) * lda + ca <= b || b + (wide_t)(nb - 1) * ldb + cb <= a) return false;
  if (lda == ldb && lda && na > 1 && nb > 1) {   // columns of one wider matrix
    const size_t d = (size_t)((b + (wide_t)lda * ((a - (a < b ? a : b)) / lda + 1) - a) % lda);
    if (ca <= d && d + cb <= lda) return false;
  }
  if (na > nb) return rows_overlap(b, nb, ldb, cb, a, na, lda, ca);
  for (size_t i = 0; i < na; i++) {   // the first row of b that ends behind row i's start
    const wide_t r = a + (wide_t)i * lda;
    const wide_t j = r < b + cb ? 0 : (ldb ? (r - b - cb) / ldb + 1 : nb);
    if (j < nb && b + j * ldb < r + ca) return true;
  }
  return false;
}

inline bool mem_overlap(const MemRows& a, const MemRows& b) {
  auto none = [](const MemRows& m) { return !m.p || !m.groups || !m.rows || !m.bytes; };
  if (none(a) || none(b)) return false;
  const wide_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  auto end = [](const MemRows& m, wide_t p) { return p + (wide_t)(m.groups - 1) * m.stride + (wide_t)(m.rows - 1) * m.ld + m.bytes; };
  if (end(a, pa) <= pb || end(b, pb) <= pa) return false;
  for (size_t i = 0; i < a.groups; i++)
    for (size_t j = 0; j < b.groups; j++)
      if (rows_overlap(pa + (wide_t)i * a.stride, a.rows, a.ld, a.bytes, pb + (wide_t)j * b.stride, b.rows, b.ld, b.bytes))
        return true;
  return false;
}

// out against each of the others.
inline int check_apart(const MemRows& out, std::initializer_list<MemRows> others) {
  for (const MemRows& m : others)
    if (mem_overlap(out, m)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s overlaps %s", out.name, m.name);
  return EXMOE_OK;
}

}  // namespace exmoe
