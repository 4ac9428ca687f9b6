// Rows and weight matrices as e4m3 values with fp32 scales (fp8.h), gfx950.
//
//   rows      v = x[r, :]                              as it is
//             v = silu(x[r, 0..n)) * x[r, n..2n)       gate and up of an expert layer side by side (silu is zero
//                                                      from -87.4 down, as the reciprocal of more than 2^126 is)
//             scales per row and 128 columns, times the row's routing weight on request: the down
//             product is linear, so a weight in the scale of its input weights its output
//   matrices  scales per 128 x 128 block
// Both are bound by memory: each element is read and written once (gate and up of 16384 rows, 84 MB, in 15 us,
// 5.5 TB/s; 128 rows in 2.6 us, the latency of one load and one store; weights of 64 experts of 2048 x 2048 in bf16,
// 805 MB, in 161 us, 5.0 TB/s, 8 of 14336 x 4096 255, 5.5 TB/s, from fp32 418, 5.6 TB/s).
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

static int quant_rows(const char* what, const exmoe_fp8_rows* call, bool gated, hipStream_t stream) {
  EXMOE_CALL(call);
  const exmoe_fp8_rows& c = *call;
  const int rows = c.rows, n = c.n, dtype = c.dtype;
  EXMOE_TRY(check_input(n, dtype));
  if (rows < 0 || rows > (1 << 30)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^30] (got %d)", rows);
  const int groups = ceil_div(n, 128);
  if ((long long)rows * groups > (kMaxThreads / 256) * 16)
    return set_error(EXMOE_ERR_UNSUPPORTED, "%s: more groups than one launch holds", what);
  if (rows == 0) return EXMOE_OK;
  const int cols = gated ? 2 * n : n, b = dtype_bytes(dtype);
  EXMOE_TRY(check_matrix("x", c.x, c.ldx, cols, b));
  EXMOE_TRY(check_matrix("q", c.q, c.ldq, n, 1));
  EXMOE_TRY(check_matrix("scale", c.scale, c.lds, groups, 4));
  EXMOE_TRY(check_int32("weights", c.weights, true));
  EXMOE_TRY(check_int32("row_index", c.row_index, true));
  if (!c.weights && c.row_index) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "row_index without weights");
  if (c.weights && c.n_weights < (c.row_index ? 1 : rows))
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%d weights, at least %d needed", c.n_weights, c.row_index ? 1 : rows);
  const MemRows mx = mem_matrix("x", c.x, rows, c.ldx, cols, b), mq = mem_matrix("q", c.q, rows, c.ldq, n, 1),
                ms = mem_matrix("scale", c.scale, rows, c.lds, groups, 4),
                mw = mem_flat("weights", c.weights, (size_t)(c.row_index ? c.n_weights : rows) * 4),
                mi = mem_flat("row_index", c.row_index, (size_t)rows * 4);
  EXMOE_TRY(check_apart(mq, {mx, mw, mi, ms}));
  EXMOE_TRY(check_apart(ms, {mx, mw, mi}));
  QuantRows a{};
  a.x = c.x; a.ldx = c.ldx; a.rows = rows; a.n = n; a.groups = groups; a.div_mul = 0xFFFFFFFFu / (uint32_t)groups;
  a.weights = c.weights; a.row_index = c.row_index; a.n_weights = c.row_index ? c.n_weights : rows; a.q = c.q; a.ldq = c.ldq;
  a.scale = c.scale; a.lds = c.lds;
  return launched(launch_rows(a, dtype, gated, stream), what);
}

extern "C" int exmoe_quantize_fp8(const exmoe_fp8_rows* call, hipStream_t stream) {
  return quant_rows("exmoe_quantize_fp8", call, false, stream);
}

extern "C" int exmoe_swiglu_fp8(const exmoe_fp8_rows* call, hipStream_t stream) {
  return quant_rows("exmoe_swiglu_fp8", call, true, stream);
}

extern "C" int exmoe_quantize_fp8_weights(const exmoe_fp8_matrices* call, hipStream_t stream) {
  EXMOE_CALL(call);
  const exmoe_fp8_matrices& c = *call;
  const int E = c.E, N = c.N, K = c.K;
  EXMOE_TRY(check_input(K, c.dtype));
  if (E < 1 || N < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "E and N must be positive (got %d, %d)", E, N);
  const int nb = ceil_div(N, 128), kb = ceil_div(K, 128);
  if (E > 65535 || nb > 65535 || (long long)E * nb * kb > kMaxThreads / 256)
    return set_error(EXMOE_ERR_UNSUPPORTED, "exmoe_quantize_fp8_weights: more blocks than one launch holds");
  const int b = dtype_bytes(c.dtype);
  EXMOE_TRY(check_matrix("w", c.w, c.ldw, K, b));
  EXMOE_TRY(check_experts("w", c.ldw, c.w_stride, N, K, E));
  EXMOE_TRY(check_matrix("q", c.q, c.ldq, K, 1));
  EXMOE_TRY(check_experts("q", c.ldq, c.q_stride, N, K, E));
  EXMOE_TRY(check_matrix("scale", c.scale, c.lds, kb, 4));
  EXMOE_TRY(check_experts("scale", c.lds, c.s_stride, nb, kb, E));
  const MemRows mw = mem_matrices("w", c.w, E, c.w_stride, N, c.ldw, K, b), mq = mem_matrices("q", c.q, E, c.q_stride, N, c.ldq, K, 1),
                ms = mem_matrices("scale", c.scale, E, c.s_stride, nb, c.lds, kb, 4);
  EXMOE_TRY(check_apart(mq, {mw, ms}));
  EXMOE_TRY(check_apart(ms, {mw}));
  QuantMatrices a{};
  a.w = c.w; a.ldw = c.ldw; a.w_stride = E > 1 ? c.w_stride : 0; a.N = N; a.K = K; a.q = c.q; a.ldq = c.ldq;
  a.q_stride = E > 1 ? c.q_stride : 0; a.scale = c.scale; a.lds = c.lds; a.s_stride = E > 1 ? c.s_stride : 0;
  return launched(by_dtype(c.dtype, [&](auto dt) {
                    ProfScope prof("quantize_fp8_weights", stream);
                    EXMOE_LAUNCH(prof, (quant_matrix_kernel<decltype(dt)::value>), dim3(kb, nb, E), dim3(256), 0, stream, a);
                    return hipGetLastError();
                  }),
                  "exmoe_quantize_fp8_weights");
}
