// Products of 8-bit operands with block scales, grouped by expert over ragged segments, gfx950.
//
//   y[s, n] = sum_b xs[src(s), b] ws[e, n / 128, b] sum_{k in block b} x[src(s), k] w[e, n, k]
//
// with blocks b of 128 summed positions, e4m3 operands and fp32 scales. A block is one matrix
// instruction (16 x 16 outputs, 128 summed positions) whose result is scaled into the fp32 sum: one
// multiply-add per output and block beside 128 products on the matrix unit.
//
// Precision. The 8-bit matrix instruction adds the products of 8 neighbouring positions with bits
// below 2^-13 of the largest of them cut off, and sums those in fp32: an output is off by at most 7 2^-13 of the
// largest product of each 8, which may exceed its rounding (256 x 256 beside seven of 3.75 x 2, in fp16: 4096
// instead of 4100) or, where products cancel, the output. On normal values it is 1.6e-5 of the result's norm, a
// hundredth of a bf16 output's rounding (1.7e-3) and a tenth of fp16's (2.1e-4). 32-bit outputs would show it there
// too, so they are made of bf16 matrix instructions (e4m3 is exact in bf16, and so are their products in fp32):
// 1e-7, at half the matrix rate.
#include "checks.h"
#include "exmoe.h"
#include "gemm_wide.h"
#include "overlap.h"
#include "row_tiles.h"

namespace exmoe {

struct Fp8Args {
  const uint8_t *x, *w;
  size_t ldx, ldw, w_stride;        // bytes
  const float *xs, *ws;
  size_t ldxs, ldws, ws_stride;     // elements
  const int32_t* offsets;           // [E + 1], or null: one matrix for all rows
  const int32_t* row_index;
  int row_div, x_rows;
  int rows, N, K, E;
  void* out;
  size_t ldo;
  int vec;
  int far;                          // rows of x behind row_index lie further apart than 32-bit offsets reach
};

typedef int i32x8 __attribute__((ext_vector_type(8)));

// A lane's 32 bytes of a 16-row fragment, 128 positions deep: row l % 16, 16-byte chunks l / 16 and
// 4 + l / 16 (any assignment of positions will do that is the same for both operands).
struct FragF8 {
  i32x8 v;
};
struct FragBF16 {
  bf16x8 v[4];
};
// Where a lane finds its two chunks of a fragment behind its first row (whose number is a multiple
// of 16: the swizzle of WideRows is then the lane's own).
struct FragPlace {
  uint32_t lo, hi;   // bytes
  __device__ __forceinline__ explicit FragPlace(int lane, int first_row) {
    const int row = lane & 15;
    lo = (first_row + row) * 128 + 16 * ((lane >> 4) ^ (row >> 1));
    hi = lo ^ 64;
  }
};
__device__ __forceinline__ FragF8 read_frag(FragF8*, const uint16_t* lds, int r0, FragPlace at) {
  const char* p = reinterpret_cast<const char*>(lds) + 128 * r0;
  const i32x4 a = *reinterpret_cast<const i32x4*>(p + at.lo), b = *reinterpret_cast<const i32x4*>(p + at.hi);
  return {__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7)};
}
__device__ __forceinline__ FragBF16 read_frag(FragBF16*, const uint16_t* lds, int r0, FragPlace at) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const i32x8 f = read_frag((FragF8*)nullptr, lds, r0, at).v;
  FragBF16 r;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    i32x4 o;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      o[2 * j] = __builtin_bit_cast(int, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)f[2 * i + j], 1.f, false));
      o[2 * j + 1] = __builtin_bit_cast(int, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)f[2 * i + j], 1.f, true));
    }
    r.v[i] = __builtin_bit_cast(bf16x8, o);
  }
  return r;
}
// The sum over the fragments' 128 positions.
__device__ __forceinline__ f32x4 block_product(const FragF8& a, const FragF8& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_product(const FragBF16& a, const FragBF16& b) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; i++) c = mfma16(a.v[i], b.v[i], c);
  return c;
}

__device__ __forceinline__ float buf_load_f32(buf_t r, uint32_t voff, uint32_t soff) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0));
}

// Row s of the sorted order: its row of x, or -1 (a row of zeros).
__device__ __forceinline__ int source_row(const Fp8Args& a, int s, uint32_t dmul) {
  if (a.row_index) {
    const int v = a.row_index[s];
    s = v < 0 ? -1 : div_by(v, a.row_div, dmul);
  }
  return s < a.x_rows ? s : -1;
}

// The rows of x of a tile: without row_index they follow each other, and offsets are from the
// tile's first one; with it they are from x's first, which 32 bits have to span.
struct TileRows {
  buf_t x, xs;
  __device__ __forceinline__ TileRows(const Fp8Args& a, const RowTile& r) {
    const int n = r.p1 - r.p0, first = a.row_index ? 0 : r.seg0 + r.p0, rows = a.row_index ? a.x_rows : n;
    x = make_buf(a.x + (size_t)first * a.ldx, (size_t)(rows - 1) * a.ldx + a.K);
    xs = make_buf(a.xs + (size_t)first * a.ldxs, 4 * ((size_t)(rows - 1) * a.ldxs + (a.K + 127) / 128));
  }
  // row i of the tile: its number behind the buffers' first row, or -1
  __device__ __forceinline__ int row(const Fp8Args& a, const RowTile& r, int i, uint32_t dmul) const {
    if (i >= r.p1 - r.p0) return -1;
    return a.row_index ? source_row(a, r.seg0 + r.p0 + i, dmul) : i;
  }
};

// Rows of x anywhere in memory (behind row_index, 2 GiB of x and more): 64-bit addresses per lane in
// place of offsets into a buffer; the layout in LDS is that of WideRows.
template <int B, int NW>
struct FarRows {
  static constexpr int kSlots = B / (8 * NW);
  int red, wave, chunk;
  const uint8_t* row[kSlots];   // null: zeros
  template <class F>
  __device__ __forceinline__ void init(int red_, int wave_, int lane, F row_at) {
    red = red_;
    wave = wave_;
    chunk = 8 * ((lane & 7) ^ WideRows<B, NW, 64>::swz(wave * 8 + lane / 8));
#pragma unroll
    for (int i = 0; i < kSlots; i++) row[i] = row_at((i * NW + wave) * 8 + lane / 8);
  }
  __device__ __forceinline__ void stage(uint16_t* lds, int k0) const {
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      const void* src = g_zero16;
      if (k0 + chunk < red && row[i]) src = row[i] + 2 * (size_t)(k0 + chunk);
      lds_copy16(src, lds + (i * NW + wave) * 8 * 64);
    }
  }
};

// 16 TP WP x 16 TQ WQ outputs per workgroup of WP x WQ waves; 128-deep slices of both operands and
// their scales double-buffered in LDS, one barrier per slice. A slice is TP steps of TQ matrix
// instructions: step i multiplies the wave's columns, held in registers, with row block i, whose
// fragment was read a step before, and scales the results of the step before into the sums. The
// slice's one barrier comes before its last step's products: the wave then holds that step's
// fragments, so every wave is done reading the slice, and the next but one is copied over it while the
// first fragments of the next are read between those products.
// Row blocks are dealt to the WP wave rows in turn, and blocks past the tile's rows are skipped.
//
// What bounds it. 256 x 256 tiles, 8192 x 8192 x 8192: 486 us, 2.26 PFLOP/s (the installed BLAS, without block
// scales, 403); the matrix unit is busy 44% of the cycles of the compute units. Per slice
// and compute unit the LDS moves 256 KB (192 KB read as fragments, 64 KB written by the copies), 2048 cycles
// at 128 bytes each, as many as the products take. Either alone would allow twice the rate: they take turns instead
// of running side by side, since the waves of a SIMD leave the barrier together. That is this schedule, not a floor.
// With parts left out, an
// earlier state of 519 us took 487 without the scaling, 477 with copies that always hit the L2, 372-400 without
// copies, 312 without copies and scaling, 323 without copies and barrier; the products alone are 250 at 2.1 GHz.
// Few tiles of few slices (512 x 4096 x 4096: one 64 x 128 tile of 32 slices a compute unit, 33 us) wait for memory
// once per slice, 1 us: only one slice is ahead.
// Measured and dropped, against 488: 32 x 32 x 64 instructions (589), one wave per SIMD with 256 x 192 outputs
// (703: the sums do not fit beside what vector instructions can address, and move to and fro), the next columns'
// fragments read ahead (spills), 128 x 128 tiles of eight waves (746) or four (649), raised priority around the
// products (506), copies spread over more steps (no change). Rows stored straight from the sums' layout, 8 bytes
// a lane, instead of in whole lines through LDS: 14336 x 4096 with 8 experts 572 us instead of 544.
template <class ET, class Frag, int TP, int TQ, int WP, int WQ, int OCC, bool FAR>
__global__ __launch_bounds__(64 * WP * WQ, OCC) void fp8_tile_kernel(Fp8Args a, int q_tiles) {
  constexpr int NW = WP * WQ, BP = 16 * TP * WP, BQ = 16 * TQ * WQ, D = 64;   // (D: pairs of bytes)
  static_assert(BQ % 128 == 0 && 128 % (16 * TQ) == 0, "a wave's columns lie in one block of scales");
  static_assert(TP % 2 == 0, "steps in pairs");
  constexpr bool F32 = std::is_same<Frag, FragBF16>::value;
  constexpr int kMfma = TQ * (F32 ? 4 : 1);   // matrix instructions of a step
  // (separate arrays: the compiler then sees that reading one does not wait for copies into another)
  __shared__ __attribute__((aligned(16))) uint16_t s_p0[BP * D], s_p1[BP * D], s_q0[BQ * D], s_q1[BQ * D];
  // scales of the rows, then of the columns' blocks (wave w copies those of rows 64 w.. of the tile, the
  // next one those of the columns, what is left zeros, so that every wave's copies are alike)
  constexpr int kScaleCopies = (BP / 64 + NW) / NW;
  __shared__ float s_s0[64 * NW * kScaleCopies], s_s1[64 * NW * kScaleCopies];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / WQ, wq = wave % WQ;
  RowTile r;
  if (!resolve_rows<BP, 16, true>(a.offsets, a.rows, a.E, q_tiles, blockIdx.x, r)) return;
  const int q0 = BQ * r.qt, red = a.K / 2;
  const uint32_t dmul = 0xFFFFFFFFu / (uint32_t)a.row_div;
  const TileRows rows(a, r);
  std::conditional_t<FAR, FarRows<BP, NW>, WideRows<BP, NW, D>> op_p;
  WideRows<BQ, NW, D> op_q;
  if constexpr (FAR) {
    op_p.init(red, wave, lane, [&](int i) {
      const int s = rows.row(a, r, i, dmul);
      return s < 0 ? nullptr : a.x + (size_t)s * a.ldx;
    });
  } else {
    op_p.init(rows.x, red, wave, lane, [&](int i) {
      const int s = rows.row(a, r, i, dmul);
      return s < 0 ? kNowhere : (uint32_t)((size_t)s * a.ldx);
    });
  }
  const int ncols = min(BQ, a.N - q0);
  op_q.init(make_buf(a.w + (size_t)r.e * a.w_stride + (size_t)q0 * a.ldw, (size_t)(ncols - 1) * a.ldw + a.K), red, wave, lane,
            [&](int i) { return i < ncols ? (uint32_t)((size_t)i * a.ldw) : kNowhere; });
  buf_t sc_buf[kScaleCopies];
  uint32_t sc_off[kScaleCopies];
  const float* sc_far[kScaleCopies];   // (FAR: addresses in place of offsets; null: zeros)
#pragma unroll
  for (int c = 0; c < kScaleCopies; c++) {
    const int part = c * NW + wave;
    sc_buf[c] = rows.xs;
    sc_off[c] = kNowhere;
    sc_far[c] = nullptr;
    if (part < BP / 64) {
      const int s = rows.row(a, r, 64 * part + lane, dmul);
      if (s >= 0) sc_off[c] = (uint32_t)((size_t)s * a.ldxs * 4), sc_far[c] = a.xs + (size_t)s * a.ldxs;
    } else if (part == BP / 64) {
      const int nb = (ncols + 127) / 128;
      const float* ws = a.ws + (size_t)r.e * a.ws_stride + (size_t)(q0 / 128) * a.ldws;
      sc_buf[c] = make_buf(ws, 4 * ((size_t)(nb - 1) * a.ldws + (a.K + 127) / 128));
      if (lane < nb) sc_off[c] = (uint32_t)((size_t)lane * a.ldws * 4), sc_far[c] = ws + (size_t)lane * a.ldws;
    }
  }
  const int steps = (a.K + 127) / 128;
  auto stage_scales = [&](int s, float* ls) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < kScaleCopies; c++) {
      auto* dst = (__attribute__((address_space(3))) void*)(ls + 64 * (c * NW + wave));
      if constexpr (FAR) {
        const void* src = g_zero16;
        if (s < steps && sc_far[c]) src = sc_far[c] + s;
        __builtin_amdgcn_global_load_lds(src, dst, 4, 0, 0);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sc_buf[c], dst, 4, s < steps ? sc_off[c] : kNowhere, s < steps ? 4 * s : 0, 0, 0);
      }
    }
  };

  f32x4 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto block_p = [&](int i) __attribute__((always_inline)) { return 16 * (i * WP + wp); };   // first row of row block i
  int nblk = 0;                                                                              // of them hold rows
#pragma unroll
  for (int i = 0; i < TP; i++) nblk += r.p0 + block_p(i) < r.p1 ? 1 : 0;
  nblk = __builtin_amdgcn_readfirstlane(nblk);

  const FragPlace at_p(lane, 16 * wp), at_q(lane, 16 * TQ * wq);
  Frag fq[TQ], fp[2];
  float sx[2], sw = 0.f;         // scales of the row block in fp[.], and of the columns
  f32x4 part[2][TQ];             // products of a step, scaled a step later
  float part_s[2];
  // products of row block i (in fp[i & 1]); those of the step before, of row block i - 1, go into the sums
  auto multiply = [&](auto full, auto i_c) __attribute__((always_inline)) {
    constexpr int i = decltype(i_c)::value, set = i & 1, before = (i + TP - 1) % TP;
    if (decltype(full)::value || i < nblk) {
      part_s[set] = sx[set] * sw;
#pragma unroll
      for (int j = 0; j < TQ; j++) part[set][j] = block_product(fq[j], fp[set]);
    }
    if (decltype(full)::value || before < nblk) {
#pragma unroll
      for (int j = 0; j < TQ; j++)
#pragma unroll
        for (int v = 0; v < 4; v++) acc[j][before][v] += part[set ^ 1][j][v] * part_s[set ^ 1];
      // (the sums stay here: moved down past a branch, they would keep the products of a whole slice)
#pragma unroll
      for (int j = 0; j < TQ; j++) asm volatile("" : "+v"(acc[j][before]));
    }
  };
  auto read_p = [&](auto i_c, const uint16_t* lp, const float* ls) __attribute__((always_inline)) {
    constexpr int i = decltype(i_c)::value;
    fp[i & 1] = read_frag((Frag*)nullptr, lp, 16 * i * WP, at_p);
    sx[i & 1] = ls[block_p(i) + (lane & 15)];
  };
  // a step by itself: its reads, copies and multiply-adds spread between its products (without
  // these groups 8192 x 8192 x 8192 took 495-507 us instead of 488)
  auto interleave = [&](auto full, auto reads_c, auto copies_c) __attribute__((always_inline)) {
    if constexpr (decltype(full)::value) {
      constexpr int reads = decltype(reads_c)::value, copies = decltype(copies_c)::value;
#pragma unroll
      for (int j = 0; j < kMfma; j++) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        // (the next row block is read behind the first product, longer runs of reads are spread)
        const int nr = reads <= 3 ? (j == 0 ? reads : 0) : (j + 1) * reads / kMfma - j * reads / kMfma;
        const int nc = (j + 1) * copies / kMfma - j * copies / kMfma;
        for (int e = 0; e < nr; e++) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        for (int e = 0; e < nc; e++) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4 * TQ / kMfma, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // the last step of the slice before, while the first fragments of slice s are read and slice s + 1
  // (or zeros past the last one) is copied; then all but the last step of slice s
  auto slice = [&](auto full, int s, uint16_t* cp, uint16_t* cq, float* cs, uint16_t* np, uint16_t* nq, float* ns)
      __attribute__((always_inline)) {
    wait_lds();      // this wave holds its last fragments of slice s - 1
    wait_vm<0>();    // its copies of slice s have landed
    block_barrier();
    multiply(full, std::integral_constant<int, TP - 1>{});
    sw = cs[BP + wq * 16 * TQ / 128];
    read_p(std::integral_constant<int, 0>{}, cp, cs);
#pragma unroll
    for (int j = 0; j < TQ; j++) fq[j] = read_frag((Frag*)nullptr, cq, 16 * j, at_q);
    interleave(full, std::integral_constant<int, 2 * TQ + 4>{}, std::integral_constant<int, 0>{});
    auto step = [&](auto i) __attribute__((always_inline)) {
      if constexpr (decltype(i)::value + 1 < TP) {
        read_p(std::integral_constant<int, decltype(i)::value + 1>{}, cp, cs);
        multiply(full, i);
        constexpr int at = decltype(i)::value, with_p = TP > 2 ? 1 : 0, with_s = TP > 3 ? 2 : with_p;
        constexpr int copies = (at == 0 ? decltype(op_q)::kSlots : 0) + (at == with_p ? decltype(op_p)::kSlots : 0) +
                               (at == with_s ? kScaleCopies : 0);
        if constexpr (at == 0) op_q.stage(nq, (s + 1) * D);
        if constexpr (at == with_p) op_p.stage(np, (s + 1) * D);
        if constexpr (at == with_s) stage_scales(s + 1, ns);
        interleave(full, std::integral_constant<int, 3>{}, std::integral_constant<int, copies>{});
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
    step(std::integral_constant<int, 4>{});
    step(std::integral_constant<int, 5>{});
    step(std::integral_constant<int, 6>{});
  };
  auto loop = [&](auto full) __attribute__((always_inline)) {
    for (int s = 0; s < steps; s += 2) {
      slice(full, s, s_p0, s_q0, s_s0, s_p1, s_q1, s_s1);
      if (s + 1 < steps) slice(full, s + 1, s_p1, s_q1, s_s1, s_p0, s_q0, s_s0);
    }
    multiply(full, std::integral_constant<int, TP - 1>{});
#pragma unroll
    for (int j = 0; j < TQ; j++)
#pragma unroll
      for (int v = 0; v < 4; v++) acc[j][TP - 1][v] += part[(TP - 1) & 1][j][v] * part_s[(TP - 1) & 1];
  };
  op_q.stage(s_q0, 0);
  op_p.stage(s_p0, 0);
  stage_scales(0, s_s0);
#pragma unroll
  for (int b = 0; b < 2; b++) {
    fp[b] = Frag{};
    sx[b] = part_s[b] = 0.f;
#pragma unroll
    for (int j = 0; j < TQ; j++) part[b][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int j = 0; j < TQ; j++) fq[j] = Frag{};
  if (nblk == TP) loop(std::true_type{});
  else loop(std::false_type{});
  wait_vm<0>();    // no copy is left behind the workgroup's end

  // Lane l holds row l % 16 and columns 4 (l / 16) + 0..3 of each 16 x 16 block: each wave turns a row block
  // at a time through its own part of LDS, so that rows leave in pieces of 16 bytes a lane, 16 TQ outputs
  // together (chunks swizzled by the row). The stores bypass the caches.
  block_barrier();   // everyone is done with the slices
  constexpr int kCols = 16 * TQ, SZ = F32 ? 4 : 2, kPitch = kCols * SZ;
  constexpr int kLanes = kPitch / 16, kRows = 64 / kLanes;   // lanes (16-byte chunks) per row, rows per store
  static_assert(16 * kPitch * NW <= (BP < BQ ? BP : BQ) * D * 4 && kLanes >= 8 && kLanes <= 16, "a block of rows per wave fits");
  char* mine = reinterpret_cast<char*>(wave < NW / 2 ? s_p0 : s_p1) + wave % (NW / 2) * 16 * kPitch;
  auto at = [&](int row, int byte) __attribute__((always_inline)) { return mine + row * kPitch + (byte ^ (16 * (row & (kLanes - 1)))); };
  const int qw = q0 + wq * kCols;
#pragma unroll
  for (int i = 0; i < TP; i++) {
    if (i >= nblk) break;
#pragma unroll
    for (int j = 0; j < TQ; j++) {
      const f32x4& c = acc[j][i];
      char* p = at(lane & 15, (16 * j + 4 * (lane >> 4)) * SZ);
      if constexpr (F32) *reinterpret_cast<f32x4*>(p) = c;
      else *reinterpret_cast<uint2*>(p) = make_uint2(ET::pack2(c[0], c[1]), ET::pack2(c[2], c[3]));
    }
    const int pb = r.p0 + block_p(i);
#pragma unroll
    for (int r0 = 0; r0 < 16; r0 += kRows) {
      const int row = r0 + lane / kLanes, col = (lane % kLanes) * (16 / SZ), q = qw + col;
      const i32x4 v = *reinterpret_cast<const i32x4*>(at(row, col * SZ));
      if (pb + row < r.p1 && q < a.N) {
        char* dst = static_cast<char*>(a.out) + ((size_t)(r.seg0 + pb + row) * a.ldo + q) * SZ;
        if (a.vec && q + 16 / SZ <= a.N) {
          __builtin_nontemporal_store(v, reinterpret_cast<i32x4*>(dst));
        } else {
#pragma unroll
          for (int e = 0; e < 16 / SZ; e++)
            if (q + e < a.N) {
              if constexpr (F32) reinterpret_cast<uint32_t*>(dst)[e] = (uint32_t)v[e];
              else reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
            }
        }
      }
    }
  }
}

// Few rows per expert, or few tiles: 16 TP rows x 16 TQ columns per workgroup, whose waves split the
// blocks of 128 positions (wave w: blocks w, w + NW, ..). Each wave copies its own slices of both operands
// into its own part of LDS, two in flight, without a barrier; the sums are added in wave order. Bound by
// reading W: 16 tokens through 64 experts of 2048 x 2048, 237 MB, in 44 us on 16 x 32 blocks of two waves
// (5.4 TB/s; a copy reaches 5.1).
template <class ET, class Frag, int TP, int TQ, int NW>
__global__ __launch_bounds__(64 * NW) void fp8_narrow_kernel(Fp8Args a, int q_tiles) {
  constexpr int D = 64, kPart = 16 * (TP + TQ) * D;
  using OpX = NarrowRows<16 * TP, D>;
  using OpW = NarrowRows<16 * TQ, D>;
  constexpr bool F32 = std::is_same<Frag, FragBF16>::value;
  __shared__ __attribute__((aligned(16))) uint16_t s_a[2][NW][kPart];
  static_assert(sizeof(f32x4) * TP * TQ * 64 * NW <= sizeof(s_a), "the sums fit into the slices' part");
  static_assert(128 % (16 * TQ) == 0, "the columns lie in one block of scales");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile r;
  if (!resolve_rows<16 * TP, 16, true>(a.offsets, a.rows, a.E, q_tiles, blockIdx.x, r)) return;
  const int n0 = 16 * TQ * r.qt, ncols = min(16 * TQ, a.N - n0), red = a.K / 2, steps = (a.K + 127) / 128;
  const uint32_t dmul = 0xFFFFFFFFu / (uint32_t)a.row_div;
  const TileRows rows(a, r);
  OpX op_x;
  OpW op_w;
  op_w.init(make_buf(a.w + (size_t)r.e * a.w_stride + (size_t)n0 * a.ldw, (size_t)(ncols - 1) * a.ldw + a.K), red, lane,
            [&](int i) { return i < ncols ? (uint32_t)((size_t)i * a.ldw) : kNowhere; });
  op_x.init(rows.x, red, lane, [&](int i) {
    const int s = rows.row(a, r, i, dmul);
    return s < 0 ? kNowhere : (uint32_t)((size_t)s * a.ldx);
  });
  uint32_t xs_off[TP];
#pragma unroll
  for (int i = 0; i < TP; i++) {
    const int s = rows.row(a, r, 16 * i + (lane & 15), dmul);
    xs_off[i] = s < 0 ? kNowhere : (uint32_t)((size_t)s * a.ldxs * 4);
  }
  const buf_t ws = make_buf(a.ws + (size_t)r.e * a.ws_stride + (size_t)(n0 / 128) * a.ldws, 4 * (size_t)steps);

  f32x4 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const FragPlace at(lane, 0);
  constexpr int kLoads = OpX::kSlots + OpW::kSlots + TP + 1;
  float sx[2][TP], sw[2];
  auto issue = [&](auto set, int n, uint16_t* lds) __attribute__((always_inline)) {
    const int b = n * NW + wave;
    op_w.stage(lds, b * D);
    op_x.stage(lds + OpW::kElems, b * D);
    const uint32_t off = b < steps ? 4 * (uint32_t)b : 0;
    sw[set] = buf_load_f32(ws, b < steps ? 0 : kNowhere, off);
#pragma unroll
    for (int i = 0; i < TP; i++) sx[set][i] = buf_load_f32(rows.xs, b < steps ? xs_off[i] : kNowhere, off);
  };
  auto compute = [&](auto set, const uint16_t* lds) __attribute__((always_inline)) {
    wait_vm<kLoads>();
    asm volatile("" ::: "memory");
    Frag fw[TQ], fx[TP];
#pragma unroll
    for (int j = 0; j < TQ; j++) fw[j] = read_frag((Frag*)nullptr, lds, 16 * j, at);
#pragma unroll
    for (int i = 0; i < TP; i++) fx[i] = read_frag((Frag*)nullptr, lds + OpW::kElems, 16 * i, at);
#pragma unroll
    for (int i = 0; i < TP; i++) {
      const float scale = sx[set][i] * sw[set];
#pragma unroll
      for (int j = 0; j < TQ; j++) {
        const f32x4 c = block_product(fw[j], fx[i]);
#pragma unroll
        for (int v = 0; v < 4; v++) acc[j][i][v] += c[v] * scale;
      }
    }
    wait_lds();   // read, before the next copies into this part
    asm volatile("" ::: "memory");
  };
  using Zero = std::integral_constant<int, 0>;
  using One = std::integral_constant<int, 1>;
  const int n = (steps + NW - 1) / NW;
  issue(Zero{}, 0, s_a[0][wave]);
  issue(One{}, 1, s_a[1][wave]);
  for (int t = 0; t < n; t += 2) {
    compute(Zero{}, s_a[0][wave]);
    issue(Zero{}, t + 2, s_a[0][wave]);
    compute(One{}, s_a[1][wave]);
    issue(One{}, t + 3, s_a[1][wave]);
  }
  wait_vm<0>();   // no copy is left behind
  __syncthreads();
  f32x4 v[TQ];
  skinny_reduce<TP, TQ, NW>(reinterpret_cast<f32x4(*)[TQ * TP][64]>(&s_a[0][0][0]), acc, wave, lane, v);
  const int p = r.p0 + 16 * wave + (lane & 15);
  if (wave >= TP || p >= r.p1) return;
#pragma unroll
  for (int j = 0; j < TQ; j++) {
    const int q = n0 + 16 * j + 4 * (lane >> 4);
    if (q < a.N) store4<ET>(a.out, (size_t)(r.seg0 + p) * a.ldo + q, F32, a.vec, a.N - q, v[j]);
  }
}

// ------------------------------------------------------------------------------------ host
template <class ET, class Frag, int TP, int TQ, int WP, int WQ, int OCC, bool FAR = false>
static hipError_t launch_tile(const Fp8Args& a, hipStream_t s) {
  constexpr int BP = 16 * TP * WP, BQ = 16 * TQ * WQ;
  const int qt = ceil_div(a.N, BQ);
  ProfScope prof("grouped_mm_fp8", s);
  EXMOE_LAUNCH(prof, (fp8_tile_kernel<ET, Frag, TP, TQ, WP, WQ, OCC, FAR>), dim3((unsigned)(row_tiles(a.rows, a.E, BP) * qt)),
               dim3(64 * WP * WQ), 0, s, a, qt);
  return hipGetLastError();
}

template <class ET, class Frag, int TP, int TQ, int NW>
static hipError_t launch_narrow(const Fp8Args& a, hipStream_t s) {
  const int qt = ceil_div(a.N, 16 * TQ);
  ProfScope prof("grouped_mm_fp8", s);
  EXMOE_LAUNCH(prof, (fp8_narrow_kernel<ET, Frag, TP, TQ, NW>), dim3((unsigned)(row_tiles(a.rows, a.E, 16 * TP) * qt)), dim3(64 * NW),
               0, s, a, qt);
  return hipGetLastError();
}

static bool few_rows(int rows, int E) { return rows <= 12 * (long long)E; }   // (16 x 32 blocks; figures below)

// Tiles of bp rows into which the experts' rows fall, on average over their remainders.
static double mean_tiles(int rows, int E, int bp) { return E > 1 ? (double)rows / bp + 0.5 * (E < rows ? E : rows) : ceil_div(rows, bp); }

// Form of the call. Measured, us (bf16 out, replayed, 512 MB of weights in turn; forms: 16 x 32 blocks / 16 x 64
// blocks / 64 x 128 tiles / 128 x 128 / 192 x 256 / 256 x 256), N x K and E experts of R rows on average:
//   2048 x 2048, E = 64, R = 2       45 /  46 /  53 /  53 /   - /   -
//                        R = 8       56 /  56 /  56 /  58 /   - /   -
//                        R = 16      64 /  60 /  58 /  58 /  63 /  65
//                        R = 32      88 /  80 /  59 /  61 /  65 /  67
//                        R = 64     135 / 116 /  69 /  64 /  67 /  68
//                        R = 256 (skewed)  - / 351 / 151 / 138 / 122 / 132
//   1024 x 2048, E = 4,  R = 125     11 /  11 /  19 /  22 /  28 /  29
//   4096 x 4096, E = 1,  R = 128      - /  16 /  33 /  39 /  53 /  56
//                        R = 512     51 /  44 /  33 /  38 /  56 /  66
//   2048 x 2048, E = 1,  R = 2048    51 /  44 /  19 /  21 /  29 /  29
//   4096 x 4096, E = 8,  R = 1024     - / 530 / 222 / 205 / 173 / 188
//   4096 x 4096, E = 1,  R = 4096     - /   - / 106 /  89 /  97 /  69
//   14336 x 4096, E = 8, R = 1024     - /   - /   - / 675 / 600 / 539
//   8192 x 8192, E = 1,  R = 8192     - /   - /   - / 643 / 554 / 486
// (fp32 out, 14336 x 4096, E = 8, R = 1024: 64 x 128 1262, 128 x 128 964) and of the blocks, two waves / four:
//   16 x 32: 4096 x 4096, E = 1, R = 1 (128 blocks)    10.9 /  8.8
//            2048 x 2048, E = 8, 2 rows (128)           6.7 /  6.1
//            2048 x 1024, E = 8, 8 rows (512)           6.6 /  6.6
//            2048 x 2048, E = 64, R = 2 (4608)         44.7 / 48.4
//            2048 x 4096, E = 64, R = 2 (4608)         90.3 / 82.9
//            4096 x 14336, E = 8, R = 1 (1024)         59.1 / 60.3
//   16 x 64: 4096 x 4096, E = 1, R = 64 (320)          13.7 / 11.6
//            2048 x 8192, E = 1, R = 128 (288)         21.6 / 16.5
//            1024 x 1024, E = 1, R = 256 (272)          5.8 /  5.8
//            1024 x 4096, E = 4, R = 125 (560)         16.5 / 16.7
//            4096 x 8192, E = 1, R = 128 (576)         27.1 / 26.6
// (K >= 4096 with few rows takes four waves throughout, 2% the worse for 4096 x 14336.)
// Few rows per expert are bound by reading W; then the number of tiles decides how many compute units work, and
// then how often the tiles fill them: 192 x 256 tiles take 0.8 of the time of 256 x 256 ones, and the last round
// of tiles is half full on average (with one expert their number is known).
template <class ET, class Frag>
static hipError_t launch_fp8(const Fp8Args& a, hipStream_t s) {
  const int E = a.E < a.rows ? a.E : a.rows;
  const long long tiles = (a.rows / 128 + (long long)E) * ceil_div(a.N, 128);
  if (a.far) return launch_tile<ET, Frag, 4, 4, 2, 2, 2, true>(a, s);
  // (four waves instead of two in a block where a compute unit has few blocks, or a block of few rows many slices)
  auto few_blocks = [&](int bq) { return a.K >= 2048 && row_tiles(a.rows, a.E, 16) * ceil_div(a.N, bq) <= 384; };
  if (few_rows(a.rows, a.E)) {
    if (a.K >= 4096 || few_blocks(32)) return launch_narrow<ET, Frag, 1, 2, 4>(a, s);
    return launch_narrow<ET, Frag, 1, 2, 2>(a, s);
  }
  if (tiles < 128) {
    if (few_blocks(64)) return launch_narrow<ET, Frag, 1, 4, 4>(a, s);
    return launch_narrow<ET, Frag, 1, 4, 2>(a, s);
  }
  if (tiles < 512 || a.rows <= 48 * (long long)a.E) return launch_tile<ET, Frag, 2, 4, 2, 2, 2>(a, s);
  if constexpr (std::is_same<Frag, FragF8>::value) {
    const int qt = ceil_div(a.N, 256);
    if (a.rows / a.E >= 160 && (long long)(a.rows / 256) * qt >= 200) {
      auto rounds = [&](int bp) { return a.E > 1 ? mean_tiles(a.rows, a.E, bp) * qt / 256 + 0.5 : (double)ceil_div((int)(mean_tiles(a.rows, 1, bp) * qt), 256); };
      if (0.8 * rounds(192) < rounds(256)) return launch_tile<ET, Frag, 6, 4, 2, 4, 2>(a, s);
      return launch_tile<ET, Frag, 8, 4, 2, 4, 2>(a, s);
    }
  }
  return launch_tile<ET, Frag, 4, 4, 2, 2, 2>(a, s);
}

}  // namespace exmoe

using namespace exmoe;

// ------------------------------------------------------------------------------------ C ABI
static int check_fp8(const char* name, const void* p, size_t ld, int K) {
  EXMOE_TRY(check_matrix(name, p, ld, K, 16));
  if (ld % 16) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: rows must be 16-byte aligned (stride %zu)", name, ld);
  if (ld > (1u << 22)) return set_error(EXMOE_ERR_UNSUPPORTED, "%s: row stride %zu, at most 2^22 is supported", name, ld);
  return EXMOE_OK;
}

extern "C" int exmoe_grouped_mm_fp8(const exmoe_grouped_fp8* call, hipStream_t stream) {
  EXMOE_CALL(call);
  const auto& [x, ldx, x_scale, ldxs, row_index, expert_offsets, w, ldw, w_stride, w_scale, ldws, ws_stride, y, ldy, x_rows, row_div,
               rows, N, K, E, out_dtype] = *call;
  if (rows < 0 || rows > (1 << 30)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^30] (got %d)", rows);
  if (N < 1 || K < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "N and K must be positive (got %d, %d)", N, K);
  if (K % 16) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "K must be a multiple of 16 (got %d)", K);
  if (N > (1 << 24) || K > (1 << 22)) return set_error(EXMOE_ERR_UNSUPPORTED, "N must be <= 2^24 and K <= 2^22");
  if (E < 1 || E > kMaxExperts) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "E must be in [1, 256] (got %d)", E);
  if (out_dtype < EXMOE_DTYPE_BF16 || out_dtype > EXMOE_DTYPE_FP32)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "out_dtype must be bf16, fp16 or fp32 (got %d)", out_dtype);
  if (row_div < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "row_div must be positive (got %d)", row_div);
  if (!expert_offsets && E > 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "expert_offsets must not be NULL with %d experts", E);
  if (rows == 0) return EXMOE_OK;
  if (x_rows < (row_index ? 1 : rows))
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "x has %d rows, at least %d needed", x_rows, row_index ? 1 : rows);
  const int ob = out_dtype == EXMOE_DTYPE_FP32 ? 4 : 2, kb = ceil_div(K, 128), nb = ceil_div(N, 128);
  EXMOE_TRY(check_fp8("x", x, ldx, K));
  EXMOE_TRY(check_fp8("w", w, ldw, K));
  EXMOE_TRY(check_experts("w", ldw, w_stride, N, K, E));
  if (E > 1 && w_stride % 16) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "w: experts must be 16-byte aligned (stride %zu)", w_stride);
  EXMOE_TRY(check_matrix("x_scale", x_scale, ldxs, kb, 4));
  EXMOE_TRY(check_matrix("w_scale", w_scale, ldws, kb, 4));
  EXMOE_TRY(check_experts("w_scale", ldws, ws_stride, nb, kb, E));
  if (ldxs > (1u << 20) || ldws > (1u << 20))
    return set_error(EXMOE_ERR_UNSUPPORTED, "x_scale, w_scale: row strides %zu and %zu, at most 2^20 is supported", ldxs, ldws);
  EXMOE_TRY(check_matrix("y", y, ldy, N, ob));
  EXMOE_TRY(check_int32("row_index", row_index, true));
  EXMOE_TRY(check_int32("expert_offsets", expert_offsets, true));
  if (!tiles_fit(rows, N, E, 64, 128, 256) || (few_rows(rows, E) && !tiles_fit(rows, N, E, 16, 32, 256)))
    return set_error(EXMOE_ERR_UNSUPPORTED, "exmoe_grouped_mm_fp8: more output tiles than one launch holds");
  const int xr = row_index ? x_rows : rows;
  const MemRows mx = mem_matrix("x", x, xr, ldx, K, 1), mw = mem_matrices("w", w, E, w_stride, N, ldw, K, 1),
                mxs = mem_matrix("x_scale", x_scale, xr, ldxs, kb, 4), mws = mem_matrices("w_scale", w_scale, E, ws_stride, nb, ldws, kb, 4),
                mi = mem_flat("row_index", row_index, (size_t)rows * 4), mo = mem_flat("expert_offsets", expert_offsets, (E + 1) * 4);
  EXMOE_TRY(check_apart(mem_matrix("y", y, rows, ldy, N, ob), {mx, mw, mxs, mws, mi, mo}));
  Fp8Args a{};
  a.x = x; a.w = w; a.ldx = ldx; a.ldw = ldw; a.w_stride = E > 1 ? w_stride : 0; a.xs = x_scale; a.ws = w_scale; a.ldxs = ldxs;
  a.ldws = ldws; a.ws_stride = E > 1 ? ws_stride : 0; a.offsets = expert_offsets; a.row_index = row_index; a.row_div = row_div;
  a.x_rows = xr; a.rows = rows; a.N = N; a.K = K; a.E = E; a.out = y; a.ldo = ldy; a.vec = vec_store(y, ldy, 0, ob == 4);
  a.far = row_index && ((size_t)x_rows * ldx >= kMaxSpan || (size_t)x_rows * ldxs * 4 >= kMaxSpan);
  const hipError_t e = out_dtype == EXMOE_DTYPE_FP32 ? launch_fp8<ElemBF16, FragBF16>(a, stream)
                       : out_dtype == EXMOE_DTYPE_FP16 ? launch_fp8<ElemFP16, FragF8>(a, stream)
                                                       : launch_fp8<ElemBF16, FragF8>(a, stream);
  return launched(e, "exmoe_grouped_mm_fp8");
}
