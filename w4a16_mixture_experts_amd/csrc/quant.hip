// Rows and weight matrices as e4m3 values with fp32 scales (fp8.h), gfx950.
//
//   rows      v = x[r, :]                              as it is
//             v = silu(x[r, 0..n)) * x[r, n..2n)       gate and up of an expert layer side by side
//             scales per row and 128 columns, times the row's routing weight on request: the down
//             product is linear, so a weight in the scale of its input weights its output
//   matrices  scales per 128 x 128 block
// Both are bound by memory: each element is read and written once.
#include "checks.h"
#include "exmoe.h"
#include "fp8.h"
#include "overlap.h"
#include "row_tiles.h"

namespace exmoe {

struct QuantRows {
  const void* x;
  size_t ldx;
  int rows, n, groups;       // groups = ceil(n / 128)
  uint32_t div_mul;          // for the division by groups
  const float* weights;      // [n_weights] or null
  const int32_t* row_index;  // [rows] or null: the row's weight is weights[row_index[r]], else weights[r]
  int n_weights;
  uint8_t* q;
  size_t ldq;
  float* scale;
  size_t lds;
};

// 16 lanes per group of 128 columns.
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantRows a) {
  const size_t task = ((size_t)blockIdx.x * 256 + threadIdx.x) / 16;
  if (task >= (size_t)a.rows * a.groups) return;   // (whole groups of 16 lanes)
  const int r = div_by((int)task, a.groups, a.div_mul), g = (int)task - r * a.groups;
  const int c = 128 * g + 8 * (threadIdx.x & 15), left = a.n - c;
  const size_t off = (size_t)r * a.ldx + c;
  f32x8 v = load_upto8<DT>(a.x, off, left);
  if constexpr (GATED) {
    const f32x8 u = load_upto8<DT>(a.x, off + a.n, left);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = silu_mul(v[i], u[i]);
  }
  const float scale = f8_scale(row16_max_u32(abs_bits8(v)));
  if (left > 0) f8_store(a.q + (size_t)r * a.ldq + c, left, f8_pack8(v, 1.f / scale));
  if ((threadIdx.x & 15) == 0) {
    float w = 1.f;
    if (a.weights) {
      const int i = a.row_index ? a.row_index[r] : r;
      w = i >= 0 && i < a.n_weights ? a.weights[i] : 0.f;
    }
    a.scale[(size_t)r * a.lds + g] = scale * w;
  }
}

struct QuantMatrices {
  const void* w;
  size_t ldw, w_stride;
  int N, K;
  uint8_t* q;
  size_t ldq, q_stride;
  float* scale;
  size_t lds, s_stride;
};

// One 128 x 128 block per workgroup: 16 lanes per row, 16 rows at a time.
template <int DT>
__global__ __launch_bounds__(256) void quant_matrix_kernel(QuantMatrices a) {
  __shared__ uint32_t s_max[4];
  const int kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
  const int c = 128 * kb + 8 * (threadIdx.x & 15), left = a.K - c, r0 = 128 * nb + threadIdx.x / 16;
  const char* w = static_cast<const char*>(a.w) + (size_t)e * a.w_stride * Elems<DT>::kBytes;
  f32x8 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int r = r0 + 16 * i;
    v[i] = load_upto8<DT>(w, (size_t)r * a.ldw + c, r < a.N ? left : 0);
    m = max(m, abs_bits8(v[i]));
  }
  m = wave_max_u32(m);
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x / 64] = m;
  __syncthreads();
  const float scale = f8_scale(max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]))), inv = 1.f / scale;
  uint8_t* q = a.q + (size_t)e * a.q_stride;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int r = r0 + 16 * i;
    if (r < a.N && left > 0) f8_store(q + (size_t)r * a.ldq + c, left, f8_pack8(v[i], inv));
  }
  if (threadIdx.x == 0) a.scale[(size_t)e * a.s_stride + (size_t)nb * a.lds + kb] = scale;
}

// ------------------------------------------------------------------------------------ host
static hipError_t launch_rows(const QuantRows& a, int dtype, bool gated, hipStream_t s) {
  const unsigned blocks = (unsigned)(((size_t)a.rows * a.groups + 15) / 16);
  return by_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    ProfScope prof(gated ? "swiglu_fp8" : "quantize_fp8", s);
    if (gated) EXMOE_LAUNCH(prof, (quant_rows_kernel<DT, true>), dim3(blocks), dim3(256), 0, s, a);
    else EXMOE_LAUNCH(prof, (quant_rows_kernel<DT, false>), dim3(blocks), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace exmoe

using namespace exmoe;

// ------------------------------------------------------------------------------------ C ABI
static int check_input(int n, int dtype) {
  if (n < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "a row must have at least one column (got %d)", n);
  if (n > (1 << 24)) return set_error(EXMOE_ERR_UNSUPPORTED, "rows must have at most 2^24 columns");
  if (dtype < EXMOE_DTYPE_BF16 || dtype > EXMOE_DTYPE_FP32)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "dtype must be bf16, fp16 or fp32 (got %d)", dtype);
  return EXMOE_OK;
}

static int quant_rows(const char* what, const void* x, size_t ldx, const float* weights, int n_weights,
                      const int32_t* row_index, int rows, int n, int dtype, bool gated, uint8_t* q, size_t ldq, float* scale,
                      size_t lds, hipStream_t stream) {
  EXMOE_TRY(check_input(n, dtype));
  if (rows < 0 || rows > (1 << 30)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^30] (got %d)", rows);
  const int groups = ceil_div(n, 128);
  if ((long long)rows * groups > (kMaxThreads / 256) * 16)
    return set_error(EXMOE_ERR_UNSUPPORTED, "%s: more groups than one launch holds", what);
  if (rows == 0) return EXMOE_OK;
  const int cols = gated ? 2 * n : n, b = dtype_bytes(dtype);
  EXMOE_TRY(check_matrix("x", x, ldx, cols, b));
  EXMOE_TRY(check_matrix("q", q, ldq, n, 1));
  EXMOE_TRY(check_matrix("scale", scale, lds, groups, 4));
  EXMOE_TRY(check_int32("weights", weights, true));
  EXMOE_TRY(check_int32("row_index", row_index, true));
  if (!weights && row_index) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "row_index without weights");
  if (weights && n_weights < (row_index ? 1 : rows))
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%d weights, at least %d needed", n_weights, row_index ? 1 : rows);
  const MemRows mx = mem_matrix("x", x, rows, ldx, cols, b), mq = mem_matrix("q", q, rows, ldq, n, 1),
                ms = mem_matrix("scale", scale, rows, lds, groups, 4),
                mw = mem_flat("weights", weights, (size_t)(row_index ? n_weights : rows) * 4),
                mi = mem_flat("row_index", row_index, (size_t)rows * 4);
  EXMOE_TRY(check_apart(mq, {mx, mw, mi, ms}));
  EXMOE_TRY(check_apart(ms, {mx, mw, mi}));
  QuantRows a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.n = n; a.groups = groups; a.div_mul = 0xFFFFFFFFu / (uint32_t)groups;
  a.weights = weights; a.row_index = row_index; a.n_weights = row_index ? n_weights : rows; a.q = q; a.ldq = ldq;
  a.scale = scale; a.lds = lds;
  return launched(launch_rows(a, dtype, gated, stream), what);
}

extern "C" int exmoe_quantize_fp8(const void* x, size_t ldx, int rows, int K, int dtype, uint8_t* q, size_t ldq, float* scale,
                                  size_t lds, hipStream_t stream) {
  return quant_rows("exmoe_quantize_fp8", x, ldx, nullptr, 0, nullptr, rows, K, dtype, false, q, ldq, scale, lds, stream);
}

extern "C" int exmoe_swiglu_fp8(const void* gate_up, size_t ldx, const float* weights, int n_weights, const int32_t* row_index,
                                int rows, int I, int dtype, uint8_t* q, size_t ldq, float* scale, size_t lds,
                                hipStream_t stream) {
  return quant_rows("exmoe_swiglu_fp8", gate_up, ldx, weights, n_weights, row_index, rows, I, dtype, true, q, ldq, scale, lds,
                    stream);
}

extern "C" int exmoe_quantize_fp8_weights(const void* w, size_t ldw, size_t w_stride, int E, int N, int K, int dtype, uint8_t* q,
                                          size_t ldq, size_t q_stride, float* scale, size_t lds, size_t s_stride,
                                          hipStream_t stream) {
  EXMOE_TRY(check_input(K, dtype));
  if (E < 1 || N < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "E and N must be positive (got %d, %d)", E, N);
  const int nb = ceil_div(N, 128), kb = ceil_div(K, 128);
  if (E > 65535 || nb > 65535 || (long long)E * nb * kb > kMaxThreads / 256)
    return set_error(EXMOE_ERR_UNSUPPORTED, "exmoe_quantize_fp8_weights: more blocks than one launch holds");
  const int b = dtype_bytes(dtype);
  EXMOE_TRY(check_matrix("w", w, ldw, K, b));
  EXMOE_TRY(check_experts("w", ldw, w_stride, N, K, E));
  EXMOE_TRY(check_matrix("q", q, ldq, K, 1));
  EXMOE_TRY(check_experts("q", ldq, q_stride, N, K, E));
  EXMOE_TRY(check_matrix("scale", scale, lds, kb, 4));
  EXMOE_TRY(check_experts("scale", lds, s_stride, nb, kb, E));
  const MemRows mw = mem_matrices("w", w, E, w_stride, N, ldw, K, b), mq = mem_matrices("q", q, E, q_stride, N, ldq, K, 1),
                ms = mem_matrices("scale", scale, E, s_stride, nb, lds, kb, 4);
  EXMOE_TRY(check_apart(mq, {mw, ms}));
  EXMOE_TRY(check_apart(ms, {mw}));
  QuantMatrices a{};
  a.w = w; a.ldw = ldw; a.w_stride = E > 1 ? w_stride : 0; a.N = N; a.K = K; a.q = q; a.ldq = ldq; a.q_stride = E > 1 ? q_stride : 0;
  a.scale = scale; a.lds = lds; a.s_stride = E > 1 ? s_stride : 0;
  return launched(by_dtype(dtype, [&](auto dt) {
                    ProfScope prof("quantize_fp8_weights", stream);
                    EXMOE_LAUNCH(prof, (quant_matrix_kernel<decltype(dt)::value>), dim3(kb, nb, E), dim3(256), 0, stream, a);
                    return hipGetLastError();
                  }),
                  "exmoe_quantize_fp8_weights");
}
