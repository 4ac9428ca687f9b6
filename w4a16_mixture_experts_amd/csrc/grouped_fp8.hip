// Products of 8-bit operands with block scales, grouped by expert over ragged segments, gfx950.
//
//   y[s, n] = sum_b xs[src(s), b] ws[e, n / 128, b] sum_{k in block b} x[src(s), k] w[e, n, k]
//
// with blocks b of 128 summed positions, e4m3 operands and fp32 scales. A block is one matrix
// instruction (16 x 16 outputs, 128 summed positions) whose result is scaled into the fp32 sum: one
// multiply-add per output and block beside 128 products on the matrix unit.
//
// Precision. The 8-bit matrix instruction adds the products of 8 neighbouring positions with bits
// below 2^-13 of the largest of them cut off, and sums those in fp32: 1.6e-5 of the result's norm
// on normal values, a hundredth of a bf16 output's rounding (2e-3) and a tenth of fp16's (2e-4).
// 32-bit outputs would show it, so they are made of bf16 matrix instructions (e4m3 is exact in bf16,
// and so are their products in fp32): 1e-7, at half the matrix rate.
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
__device__ __forceinline__ FragF8 read_frag(FragF8*, const uint16_t* lds, int r0, int lane) {
  const i32x4 a = __builtin_bit_cast(i32x4, NarrowRows<16, 64>::frag(lds, r0, 0, lane));
  const i32x4 b = __builtin_bit_cast(i32x4, NarrowRows<16, 64>::frag(lds, r0, 1, lane));
  return {__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7)};
}
__device__ __forceinline__ FragBF16 read_frag(FragBF16*, const uint16_t* lds, int r0, int lane) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const i32x8 f = read_frag((FragF8*)nullptr, lds, r0, lane).v;
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

// 16 TP WP x 16 TQ WQ outputs per workgroup of WP x WQ waves; 128-deep slices of both operands
// double-buffered in LDS, one barrier per slice.
template <class ET, class Frag, int TP, int TQ, int WP, int WQ, int OCC>
__global__ __launch_bounds__(64 * WP * WQ, OCC) void fp8_tile_kernel(Fp8Args a, int q_tiles) {
  constexpr int NW = WP * WQ, BP = 16 * TP * WP, BQ = 16 * TQ * WQ, D = 64;   // (D: pairs of bytes)
  static_assert(BQ % 128 == 0 && 128 % (16 * TQ) == 0, "a wave's columns lie in one block of scales");
  __shared__ __attribute__((aligned(16))) uint16_t s_p0[BP * D], s_p1[BP * D], s_q0[BQ * D], s_q1[BQ * D];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / WQ, wq = wave % WQ;
  RowTile r;
  if (!resolve_rows<BP, 16, true>(a.offsets, a.rows, a.E, q_tiles, blockIdx.x, r)) return;
  const int q0 = BQ * r.qt, red = a.K / 2;
  const uint32_t dmul = 0xFFFFFFFFu / (uint32_t)a.row_div;
  const TileRows rows(a, r);
  WideRows<BP, NW, D> op_p;
  WideRows<BQ, NW, D> op_q;
  op_p.init(rows.x, red, wave, lane, [&](int i) {
    const int s = rows.row(a, r, i, dmul);
    return s < 0 ? kNowhere : (uint32_t)((size_t)s * a.ldx);
  });
  const int ncols = min(BQ, a.N - q0);
  op_q.init(make_buf(a.w + (size_t)r.e * a.w_stride + (size_t)q0 * a.ldw, (size_t)(ncols - 1) * a.ldw + a.K), red, wave, lane,
            [&](int i) { return i < ncols ? (uint32_t)((size_t)i * a.ldw) : kNowhere; });
  uint32_t xs_off[TP];
#pragma unroll
  for (int i = 0; i < TP; i++) {
    const int s = rows.row(a, r, 16 * (i * WP + wp) + (lane & 15), dmul);
    xs_off[i] = s < 0 ? kNowhere : (uint32_t)((size_t)s * a.ldxs * 4);
  }
  const int nb = min((q0 + 16 * TQ * wq) / 128, (a.N - 1) / 128);   // (columns past N: any scale)
  const float* ws = a.ws + (size_t)r.e * a.ws_stride + (size_t)nb * a.ldws;

  f32x4 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = (a.K + 127) / 128;
  auto slice = [&](int s, const uint16_t* cp, const uint16_t* cq, uint16_t* np, uint16_t* nq) __attribute__((always_inline)) {
    float sc[TP];
    const float w = ws[s];
#pragma unroll
    for (int i = 0; i < TP; i++) sc[i] = buf_load_f32(rows.xs, xs_off[i], 4 * s) * w;
    wait_vm<0>();
    wait_lds();
    block_barrier();
    if (s + 1 < steps) {
      op_p.stage(np, (s + 1) * D);
      op_q.stage(nq, (s + 1) * D);
    }
    Frag fq[TQ];
#pragma unroll
    for (int j = 0; j < TQ; j++) fq[j] = read_frag((Frag*)nullptr, cq, (wq * TQ + j) * 16, lane);
#pragma unroll
    for (int i = 0; i < TP; i++) {
      const Frag fp = read_frag((Frag*)nullptr, cp, 16 * (i * WP + wp), lane);
#pragma unroll
      for (int j = 0; j < TQ; j++) {
        const f32x4 c = block_product(fq[j], fp);
#pragma unroll
        for (int v = 0; v < 4; v++) acc[j][i][v] += c[v] * sc[i];
      }
    }
  };
  op_p.stage(s_p0, 0);
  op_q.stage(s_q0, 0);
  for (int s = 0; s < steps; s += 2) {
    slice(s, s_p0, s_q0, s_p1, s_q1);
    if (s + 1 < steps) slice(s + 1, s_p1, s_q1, s_p0, s_q0);
  }
  // lane l holds row l % 16 and columns 4 (l / 16) + 0..3 of each 16 x 16 block
  constexpr bool F32 = std::is_same<Frag, FragBF16>::value;
#pragma unroll
  for (int i = 0; i < TP; i++) {
    const int p = r.p0 + 16 * (i * WP + wp) + (lane & 15);
    if (p >= r.p1) continue;
    const size_t row = (size_t)(r.seg0 + p) * a.ldo;
#pragma unroll
    for (int j = 0; j < TQ; j++) {
      const int q = q0 + (wq * TQ + j) * 16 + 4 * (lane >> 4);
      if (q < a.N) store4<ET>(a.out, row + q, F32, a.vec, a.N - q, acc[j][i]);
    }
  }
}

// ------------------------------------------------------------------------------------ host
template <class ET, class Frag>
static hipError_t launch_fp8(const Fp8Args& a, hipStream_t s) {
  constexpr int BP = 128, BQ = 128;
  const int qt = ceil_div(a.N, BQ);
  ProfScope prof("grouped_mm_fp8", s);
  EXMOE_LAUNCH(prof, (fp8_tile_kernel<ET, Frag, 4, 4, 2, 2, 2>), dim3((unsigned)(row_tiles(a.rows, a.E, BP) * qt)), dim3(256), 0, s,
               a, qt);
  return hipGetLastError();
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

extern "C" int exmoe_grouped_mm_fp8(const uint8_t* x, size_t ldx, const float* x_scale, size_t ldxs, int x_rows,
                                    const int32_t* row_index, int row_div, const int32_t* expert_offsets, const uint8_t* w,
                                    size_t ldw, size_t w_stride, const float* w_scale, size_t ldws, size_t ws_stride, int rows,
                                    int N, int K, int E, int out_dtype, void* y, size_t ldy, hipStream_t stream) {
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
  if (ldxs > (1u << 20)) return set_error(EXMOE_ERR_UNSUPPORTED, "x_scale: row stride %zu, at most 2^20 is supported", ldxs);
  EXMOE_TRY(check_matrix("y", y, ldy, N, ob));
  EXMOE_TRY(check_int32("row_index", row_index, true));
  EXMOE_TRY(check_int32("expert_offsets", expert_offsets, true));
  if (row_index && ((size_t)x_rows * ldx >= kMaxSpan || (size_t)x_rows * ldxs * 4 >= kMaxSpan))
    return set_error(EXMOE_ERR_UNSUPPORTED, "x of %d rows behind row_index spans 2 GiB or more", x_rows);
  if (!tiles_fit(rows, N, E, 128, 128, 256))
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
  const hipError_t e = out_dtype == EXMOE_DTYPE_FP32 ? launch_fp8<ElemBF16, FragBF16>(a, stream)
                       : out_dtype == EXMOE_DTYPE_FP16 ? launch_fp8<ElemFP16, FragF8>(a, stream)
                                                       : launch_fp8<ElemBF16, FragF8>(a, stream);
  return launched(e, "exmoe_grouped_mm_fp8");
}
