// Tiles over ragged segments of rows sorted by expert, shared by the grouped products
// (grouped.hip, grouped_fp8.hip).
#pragma once

#include "gemm_tile.h"

namespace exmoe {

struct RowTile {
  int e, seg0, cnt, p0, p1, qt;   // rows p0..p1 of the segment
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Inclusive sum over the lanes of a wave: row shifts inside 16 lanes, then the rows' totals.
__device__ __forceinline__ int wave_scan(int v) {
  auto step = [&](auto ctrl) __attribute__((always_inline)) {
    v += __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, 0xF, 0xF, true);   // row_shr: zeros shifted in
  };
  step(std::integral_constant<int, 0x111>{});
  step(std::integral_constant<int, 0x112>{});
  step(std::integral_constant<int, 0x114>{});
  step(std::integral_constant<int, 0x118>{});
  const int t0 = __builtin_amdgcn_readlane(v, 15), t1 = __builtin_amdgcn_readlane(v, 31),
            t2 = __builtin_amdgcn_readlane(v, 47);
  const int row = (int)lane_id() >> 4;
  return v + (row > 0 ? t0 : 0) + (row > 1 ? t1 : 0) + (row > 2 ? t2 : 0);
}

// Tile of workgroup b among ceil(count_e / BP) x q_tiles tiles per expert. Every wave finds
// it by itself (no barrier): lane l holds experts 4 l .. 4 l + 3. WHOLE: offsets may be null, one
// segment of all rows.
template <int BP, int BLOCK = 32, bool WHOLE = false>
__device__ __forceinline__ bool resolve_rows(const int32_t* __restrict__ offsets, int rows, int E, int q_tiles, int b,
                                             RowTile& t) {
  const int lane = (int)lane_id();
  int o[5], v[4], run = 0;
#pragma unroll
  for (int q = 0; q < 5; q++) {
    const int e = lane * 4 + q;
    o[q] = WHOLE && !offsets ? (e > 0 ? rows : 0) : offsets[e <= E ? e : E];
  }
#pragma unroll
  for (int q = 0; q < 5; q++) o[q] = clampi(o[q], 0, rows);
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const int c = lane * 4 + q < E ? o[q + 1] - o[q] : 0;
    v[q] = c > 0 ? (c + BP - 1) / BP : 0;
    run += v[q];
  }
  const int incl = wave_scan(run);
  const int total = __builtin_amdgcn_readlane(incl, 63) * q_tiles;
  if (b >= total) return false;
  const int idx = xcd_contiguous(b, total);
  // the first lane whose experts end past the tile, then the expert of the four
  const int own = __ffsll((long long)__ballot(incl * q_tiles > idx)) - 1;
  int start = __builtin_amdgcn_readlane(incl - run, own), seg0 = 0, end = 0, e = 0;
  bool found = false;
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const int vq = __builtin_amdgcn_readlane(v[q], own);
    if (!found && (start + vq) * q_tiles > idx) {
      found = true;
      e = own * 4 + q;
      seg0 = __builtin_amdgcn_readlane(o[q], own);
      end = __builtin_amdgcn_readlane(o[q + 1], own);
    }
    if (!found) start += vq;
  }
  t.e = e;
  t.seg0 = seg0;
  t.cnt = end - seg0;
  // the expert's rows are dealt evenly to its tiles, in whole blocks
  const int np = (t.cnt + BP - 1) / BP;
  int pt;
  band_order(idx - start * q_tiles, np, q_tiles, pt, t.qt);
  const int blocks = (t.cnt + BLOCK - 1) / BLOCK, each = blocks / np, more = blocks - each * np;
  t.p0 = BLOCK * (each * pt + min(pt, more));
  t.p1 = min(t.cnt, t.p0 + BLOCK * (each + (pt < more ? 1 : 0)));
  return true;
}

// value / d for 0 <= value, d >= 1, with mul = floor((2^32 - 1) / d): the high product is
// the quotient or one less, and one compare corrects it.
__device__ __forceinline__ int div_by(int v, int d, uint32_t mul) {
  uint32_t q = __umulhi((uint32_t)v, mul);
  if ((uint32_t)v - q * (uint32_t)d >= (uint32_t)d) q++;
  return (int)q;
}

// ------------------------------------------------------------------------------------ host
inline int ceil_div(int a, int b) { return (int)(((long long)a + b - 1) / b); }
constexpr long long kMaxThreads = 0xFFFFFF00ll;   // of one launch, in whole workgroups; larger calls are refused

// Tiles of BP rows, at most, into which the experts' rows fall.
inline long long row_tiles(int rows, int E, int bp) { return rows / bp + (E < rows ? E : rows); }
// Whether the bp x bq tiles of rows x Q outputs, one workgroup of that many threads each, are one launch.
inline bool tiles_fit(int rows, int Q, int E, int bp, int bq, int threads) {
  return row_tiles(rows, E, bp) * ceil_div(Q, bq) * threads <= kMaxThreads;
}

}  // namespace exmoe
