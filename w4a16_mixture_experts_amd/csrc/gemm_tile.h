// Matrix-product tiles shared by the grouped products (grouped.hip) and the projection
// with low-rank adapters (lora.hip): 16-bit operands, fp32 accumulation on MFMA.
//
// Every product here is D[p, q] = sum_r P(p, r) Q(q, r) with q contiguous in the output.
// An operand is stored either with the summed axis contiguous ("rows": one row per p or q)
// or with it outermost ("columns": one row per r, read transposed):
//   forward          p = routed row (rows), q = output (rows of W),    r = K
//   gradient of x    p = routed row (rows), q = input (columns of W),  r = N
//   gradient of W    p = output (columns),  q = input (columns),       r = routed row
// MFMA takes Q as its A operand and P as its B operand, so that a lane ends with four
// consecutive q of one p: one 8-byte (16-bit outputs) or 16-byte (fp32) store.
//
// Both operands go from memory straight into LDS (global_load_lds, 16 bytes a lane).
// LDS layout of a 64-deep slice:
//   rows:    [row][64], the 16-byte chunk c of row i at position c ^ ((i >> 1) & 7): the 16
//            rows of a fragment read (one chunk each) cover all 64 banks once;
//   columns: [64][B], the 32-byte unit u of row r at position u ^ col_swz(r): the eight
//            rows that 32 lanes of a transposing read touch cover all 64 banks once.
#pragma once

#include <type_traits>

#include "common.h"
#include "device.h"

namespace exmoe {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Element types of the operands: bf16 or fp16 bit patterns in memory.
struct ElemBF16 {
  static __device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) { return mfma16(a, b, c); }
  static __device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ uint16_t from_f32(float v) { return f32_to_bf16(v); }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) { return pack_bf16x2(lo, hi); }
};
struct ElemFP16 {
  static __device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  static __device__ __forceinline__ float to_f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t from_f32(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return (uint32_t)from_f32(lo) | ((uint32_t)from_f32(hi) << 16);
  }
};

constexpr int kBK = 64;   // depth of one staged slice

// Zero bytes: what a copy (16 of them) or Any8 (20) reads in place of elements past the
// summed axis (device globals start zeroed; never written).
static __device__ __attribute__((aligned(16))) uint16_t g_zero16[16];

__device__ __forceinline__ void lds_copy16(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

__device__ __forceinline__ int col_swz(int r) { return (r & 3) | (((r >> 3) & 1) << 2); }

// Eight elements of a row-major matrix at any alignment: element off + i of base is used when
// i < n (and ok), else it is zero. Reads only elements of the matrix. fetch() starts the
// loads, value() gives the elements. Away from the rows' ends (inner): five aligned words
// around the eight elements, shifted by one element where the address needs it (a fifth of
// the loads and a tenth of the vector instructions of loading them one by one).
struct Any8 {
  uint32_t w0, w1, w2, w3, w4, odd;
  static __device__ __forceinline__ bool inner(const uint16_t* base, size_t off, int n, bool ok) {
    // the words hold elements -1 or 0 .. 8 or 9
    return !ok || (n >= 10 && (off > 0 || ((uintptr_t)base & 2) == 0));
  }
  __device__ __forceinline__ void fetch(const uint16_t* base, size_t off, bool ok) {   // of an inner one
    const uint16_t* p = base + off;
    odd = ok ? (uint32_t)((uintptr_t)p & 2) : 0;
    typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
    const uint32_t* q = reinterpret_cast<const uint32_t*>(ok ? (uintptr_t)p & ~(uintptr_t)3 : (uintptr_t)g_zero16);
    const u32x4_a4 v = *reinterpret_cast<const u32x4_a4*>(q);
    w0 = v[0];
    w1 = v[1];
    w2 = v[2];
    w3 = v[3];
    w4 = q[4];
  }
  __device__ __forceinline__ void fetch_edge(const uint16_t* base, size_t off, int n, bool ok) {
    auto pair = [&](int j) __attribute__((always_inline)) {
      const bool u0 = ok && j < n, u1 = ok && j + 1 < n;
      const uint32_t e0 = base[u0 ? off + j : 0], e1 = base[u1 ? off + j + 1 : 0];
      return (u0 ? e0 : 0u) | (u1 ? e1 << 16 : 0u);
    };
    w0 = pair(0);
    w1 = pair(2);
    w2 = pair(4);
    w3 = pair(6);
    w4 = 0;
    odd = 0;
  }
  __device__ __forceinline__ uint4 value() const {
    return make_uint4(__builtin_amdgcn_alignbyte(w1, w0, odd), __builtin_amdgcn_alignbyte(w2, w1, odd),
                      __builtin_amdgcn_alignbyte(w3, w2, odd), __builtin_amdgcn_alignbyte(w4, w3, odd));
  }
};

// Operand stored as rows (summed axis contiguous), B rows per slice, staged by NW waves.
template <int B, int NW>
struct RowOperand {
  static constexpr int kSlots = B / 8 / NW;   // copies per lane and slice (8 rows each)
  static_assert(B % (8 * NW) == 0, "rows per slice");
  const uint16_t* base;
  size_t off[kSlots];        // element offset of the lane's row (clamped to a readable one)
  int red;                   // length of the summed axis

  // row_off(i): element offset of row i of the tile (any readable row past the end)
  template <class F>
  __device__ __forceinline__ void init(const uint16_t* b, int red_, int wave, int lane, F row_off) {
    base = b;
    red = red_;
#pragma unroll
    for (int i = 0; i < kSlots; i++) off[i] = row_off((i * NW + wave) * 8 + (lane >> 3));
  }
  __device__ __forceinline__ int column(int i, int k0, int wave, int lane) const {
    const int row = (i * NW + wave) * 8 + (lane >> 3);
    return k0 + 8 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  __device__ __forceinline__ void stage(uint16_t* lds, int k0, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      const int col = column(i, k0, wave, lane);
      uint16_t* dst = lds + (i * NW + wave) * 8 * kBK;
      const uint16_t* src = base + off[i] + col;
      if (k0 + kBK > red && col >= red) src = g_zero16;
      lds_copy16(src, dst);
    }
  }
  // any alignment: the slice's loads, and later their values to LDS
  __device__ __forceinline__ void fetch(Any8 (&r)[kSlots], int k0, int wave, int lane) const {
    bool in = true;
#pragma unroll
    for (int i = 0; i < kSlots; i++) in = in && Any8::inner(base, off[i] + column(i, k0, wave, lane), red - column(i, k0, wave, lane), true);
    if (__all(in)) {
#pragma unroll
      for (int i = 0; i < kSlots; i++) r[i].fetch(base, off[i] + column(i, k0, wave, lane), true);
    } else {
#pragma unroll
      for (int i = 0; i < kSlots; i++)
        r[i].fetch_edge(base, off[i] + column(i, k0, wave, lane), red - column(i, k0, wave, lane), true);
    }
  }
  __device__ __forceinline__ void commit(const Any8 (&r)[kSlots], uint16_t* lds, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < kSlots; i++) *reinterpret_cast<uint4*>(lds + (i * NW + wave) * 8 * kBK + 8 * lane) = r[i].value();
  }
  // fragment of rows r0..r0+15, summed positions 32 kk + 8 (lane / 16) + 0..7
  static __device__ __forceinline__ bf16x8 frag(const uint16_t* lds, int r0, int kk, int lane) {
    const int row = r0 + (lane & 15);
    const int pos = (4 * kk + (lane >> 4)) ^ ((row >> 1) & 7);
    return *reinterpret_cast<const bf16x8*>(lds + row * kBK + 8 * pos);
  }
};

// Operand stored as columns (summed axis outermost), B columns per slice.
template <int B, int NW>
struct ColOperand {
  static constexpr int kChunks = B / 8;                 // 16-byte chunks per row
  static constexpr int kRows = 64 / kChunks;            // rows per wave-wide copy
  static constexpr int kSlots = kBK / (kRows * NW);
  static_assert(B >= 128 && B <= 512 && kBK % (kRows * NW) == 0, "columns per slice");
  const uint16_t* base;      // column 0 of the tile, row 0 of the summed axis
  size_t ld;
  int red;                   // rows of the summed axis
  int ncols;                 // readable columns from base on

  __device__ __forceinline__ void init(const uint16_t* b, size_t ld_, int red_, int ncols_) {
    base = b;
    ld = ld_;
    red = red_;
    ncols = ncols_;
  }
  __device__ __forceinline__ int row_of(int i, int wave, int lane) const { return (i * NW + wave) * kRows + lane / kChunks; }
  __device__ __forceinline__ int column(int i, int wave, int lane) const {
    const int pos = lane % kChunks;
    return 16 * ((pos >> 1) ^ col_swz(row_of(i, wave, lane))) + 8 * (pos & 1);
  }
  // row_off(r, i): element offset of row r (0 <= r < red; i: the lane's slot), or ~0 for zeros
  template <class F>
  __device__ __forceinline__ void stage(uint16_t* lds, int k0, int wave, int lane, F row_off) const {
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      const int row = k0 + row_of(i, wave, lane), col = column(i, wave, lane);
      const size_t o = row < red ? row_off(row, i) : ~(size_t)0;
      const uint16_t* src = base + o + (col < ncols ? col : 0);
      if (o == ~(size_t)0) src = g_zero16;
      lds_copy16(src, lds + (i * NW + wave) * kRows * B);
    }
  }
  template <class F>
  __device__ __forceinline__ void fetch(Any8 (&r)[kSlots], int k0, int wave, int lane, F row_off) const {
    size_t o[kSlots];
    bool in = true;
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      const int row = k0 + row_of(i, wave, lane), col = column(i, wave, lane);
      o[i] = row < red ? row_off(row, i) : ~(size_t)0;
      if (col >= ncols) o[i] = ~(size_t)0;
      in = in && Any8::inner(base, o[i] + col, ncols - col, o[i] != ~(size_t)0);
    }
    if (__all(in)) {
#pragma unroll
      for (int i = 0; i < kSlots; i++) r[i].fetch(base, o[i] + column(i, wave, lane), o[i] != ~(size_t)0);
    } else {
#pragma unroll
      for (int i = 0; i < kSlots; i++)
        r[i].fetch_edge(base, o[i] + column(i, wave, lane), ncols - column(i, wave, lane), o[i] != ~(size_t)0);
    }
  }
  __device__ __forceinline__ void commit(const Any8 (&r)[kSlots], uint16_t* lds, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < kSlots; i++) *reinterpret_cast<uint4*>(lds + (i * NW + wave) * kRows * B + 8 * lane) = r[i].value();
  }
  // fragment of columns c0..c0+15, summed positions 32 kk + 8 (lane / 16) + 0..7: two
  // transposing reads, each turning a block of 4 rows x 16 columns per 16 lanes into 4
  // consecutive rows of one column per lane
  static __device__ __forceinline__ bf16x8 frag(const uint16_t* lds, int c0, int kk, int lane) {
    const int f = ((lane >> 2) & 3) | (((lane >> 4) & 1) << 2);   // col_swz of both rows read
    const int row = 32 * kk + 8 * (lane >> 4) + ((lane >> 2) & 3);
    const uint16_t* p = lds + row * B + 16 * ((c0 >> 4) ^ f) + 4 * (lane & 3);
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * B));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// Four consecutive outputs q..q+3 of a row: one wide store where the row allows it (vec),
// else element by element up to n.
template <class ET>
__device__ __forceinline__ void store4(void* out, size_t off, bool out_f32, bool vec, int n, f32x4 v) {
  if (out_f32) {
    float* o = static_cast<float*>(out) + off;
    if (vec && n >= 4) {
      *reinterpret_cast<f32x4*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (i < n) o[i] = v[i];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + off;
    if (vec && n >= 4) {
      *reinterpret_cast<uint2*>(o) = make_uint2(ET::pack2(v[0], v[1]), ET::pack2(v[2], v[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (i < n) o[i] = ET::from_f32(v[i]);
    }
  }
}

// ---- few rows, operands of any alignment: the waves of a workgroup split the summed axis in
// 32-deep steps (wave w: steps w, w + NW, ...), each lane loads its fragments as the words
// around their eight elements (Any8; row or column l % 16, positions 8 (l / 16) + 0..7).
// xrow[i] / wrow[j]: element offset of the lane's row of each block in x / w.
template <class ET, int TP, int TQ, int NW>
__device__ __forceinline__ void skinny_product_any(const uint16_t* __restrict__ x, const size_t (&xrow)[TP],
                                                   const uint16_t* __restrict__ w, const size_t (&wrow)[TQ], int red,
                                                   int wave, int lane, f32x4 (&acc)[TQ][TP]) {
  constexpr int kU = 2;   // steps whose loads are in flight together
  for (int k0 = 32 * wave; k0 < red; k0 += 32 * NW * kU) {
    Any8 rw[kU][TQ], rx[kU][TP];
    bool in = true;
#pragma unroll
    for (int u = 0; u < kU; u++) {
      const int k = k0 + 32 * NW * u + 8 * (lane >> 4);
#pragma unroll
      for (int j = 0; j < TQ; j++) in = in && Any8::inner(w, wrow[j] + k, red - k, k < red);
#pragma unroll
      for (int i = 0; i < TP; i++) in = in && Any8::inner(x, xrow[i] + k, red - k, k < red);
    }
    auto fetch_all = [&](auto inner) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < kU; u++) {
        const int k = k0 + 32 * NW * u + 8 * (lane >> 4);
#pragma unroll
        for (int j = 0; j < TQ; j++) {
          if constexpr (decltype(inner)::value) rw[u][j].fetch(w, wrow[j] + k, k < red);
          else rw[u][j].fetch_edge(w, wrow[j] + k, red - k, k < red);
        }
#pragma unroll
        for (int i = 0; i < TP; i++) {
          if constexpr (decltype(inner)::value) rx[u][i].fetch(x, xrow[i] + k, k < red);
          else rx[u][i].fetch_edge(x, xrow[i] + k, red - k, k < red);
        }
      }
    };
    if (__all(in)) fetch_all(std::true_type{});
    else fetch_all(std::false_type{});
#pragma unroll
    for (int u = 0; u < kU; u++)
#pragma unroll
      for (int j = 0; j < TQ; j++)
#pragma unroll
        for (int i = 0; i < TP; i++)
          acc[j][i] = ET::mfma(__builtin_bit_cast(bf16x8, rw[u][j].value()), __builtin_bit_cast(bf16x8, rx[u][i].value()),
                               acc[j][i]);
  }
}

// Sum over the waves in wave order: part [NW][TQ TP][64] in LDS. Wave w < TP gets those of
// row block w, v[j] of column block j.
template <int TP, int TQ, int NW>
__device__ __forceinline__ void skinny_reduce(f32x4 (*part)[TQ * TP][64], const f32x4 (&acc)[TQ][TP], int wave, int lane,
                                              f32x4 (&v)[TQ]) {
  static_assert(TP <= NW, "a wave per row block");
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) part[wave][j * TP + i][lane] = acc[j][i];
  __syncthreads();
  if (wave >= TP) return;
#pragma unroll
  for (int j = 0; j < TQ; j++) {
    v[j] = part[0][j * TP + wave][lane];
#pragma unroll
    for (int w = 1; w < NW; w++) {
      const f32x4 q = part[w][j * TP + wave][lane];
#pragma unroll
      for (int e = 0; e < 4; e++) v[j][e] += q[e];
    }
  }
}

// Workgroup b of a launch of n runs on XCD b % 8 (round-robin dispatch). This gives each
// XCD a contiguous run of the logical indices 0..n-1, so that tiles that share operand
// slices share an L2.
__device__ __forceinline__ int xcd_contiguous(int b, int n) {
  const int x = b & 7, i = b >> 3, q = n >> 3, r = n & 7;
  return x * q + (x < r ? x : r) + i;
}

// Order of the np x nq tiles of one matrix: bands of up to 8 row tiles, in a band column by
// column. The 32 tiles that run at once on an XCD are then about 8 x 4, which shares both
// operands' slices in its L2 (one row of tiles would read 33 slices a step instead of 12;
// 8192 x 8192 x 8192: 1394 -> 922 us).
__device__ __forceinline__ void band_order(int idx, int np, int nq, int& pt, int& qt) {
  constexpr int kBand = 8;
  const int band = idx / (kBand * nq), rows = min(kBand, np - band * kBand);
  idx -= band * kBand * nq;
  qt = idx / rows;
  pt = band * kBand + idx - qt * rows;
}

}  // namespace exmoe
