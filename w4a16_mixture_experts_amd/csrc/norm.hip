// Root-mean-square norm of rows with the residual's addition, in 16 or 32 bits and as e4m3 values
// with scales (fp8.h), gfx950.
//
//   h = x + residual rounded to the residual's type (what is stored is what is normed), or x
//   y[i] = h[i] / sqrt(mean(h^2) + eps) * w[i]
// in fp32; y is rounded once to x's type, and q is made of the fp32 value, not of the rounded y. Rows whose squares
// leave the range of 32 bits are scaled by a power of two first.
// Bound by memory: a row is read once, held in registers between the sum of its squares and its
// outputs, and written once (4096 x 4096, 152 MB, 25 us where the inputs are in the memory-side cache, 30 us where
// not: 5.1 TB/s, the rate of a copy).
#include "checks.h"
#include "exmoe.h"
#include "fp8.h"
#include "overlap.h"
#include "row_tiles.h"

namespace exmoe {

struct NormArgs {
  const void* x;
  size_t ldx;
  const void* w;
  const void* res;
  size_t ldr;
  void* res_out;
  size_t ldro;
  int w_f32, res_f32;        // 32 bits instead of x's type
  float eps;
  int T, H;
  void* y;
  size_t ldy;
  uint8_t* q;
  size_t ldq;
  float* scale;
  size_t lds;
};

// WAVES waves per row, each lane CH chunks of 8 columns: chunk j of thread t is j 64 WAVES + t,
// so that 16 neighbouring lanes hold 128 columns of one scale.
template <int DT, int WAVES, int CH>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void rms_norm_kernel(NormArgs a) {
  constexpr int THREADS = 64 * WAVES;
  const int t = WAVES == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int row = WAVES == 1 ? (int)(blockIdx.x * 4 + threadIdx.x / 64) : (int)blockIdx.x;
  if (row >= a.T) return;    // (a whole wave, and with several waves per row never)
  f32x8 h[CH];
  const size_t xo = (size_t)row * a.ldx;
#pragma unroll
  for (int j = 0; j < CH; j++) {
    const int c = 8 * (j * THREADS + t);
    h[j] = load_upto8<DT>(a.x, xo + c, a.H - c);
  }
  if (a.res) {               // (uniform)
    const size_t ro = (size_t)row * a.ldr, wo = (size_t)row * a.ldro;
    auto add = [&](auto rt) __attribute__((always_inline)) {
      constexpr int RT = decltype(rt)::value;
      f32x8 r[CH];
#pragma unroll
      for (int j = 0; j < CH; j++) {
        const int c = 8 * (j * THREADS + t);
        r[j] = load_upto8<RT>(a.res, ro + c, a.H - c);
      }
#pragma unroll
      for (int j = 0; j < CH; j++) {
        const int c = 8 * (j * THREADS + t);
#pragma unroll
        for (int i = 0; i < 8; i++) h[j][i] = Elems<RT>::rounded(h[j][i] + r[j][i]);
        store_upto8<RT>(a.res_out, wo + c, a.H - c, h[j]);
      }
    };
    if (a.res_f32) add(std::integral_constant<int, EXMOE_DTYPE_FP32>{});
    else add(std::integral_constant<int, DT>{});
  }
  __shared__ float s_sum[2][WAVES];
  auto squares = [&](int pass) __attribute__((always_inline)) {   // their sum over the row, in all of its lanes
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < CH; j++) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) s += h[j][i] * h[j][i];
      sum += s;
    }
    sum = wave_sum_f32(sum);
    if constexpr (WAVES > 1) {
      if ((t & 63) == 0) s_sum[pass][t / 64] = sum;
      __syncthreads();
      sum = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; w++) sum += s_sum[pass][w];
    }
    return sum;
  };
  float mean = squares(0) / (float)a.H + a.eps;
  if (!(mean >= 0x1p-80f && mean <= 0x1p100f)) {   // (uniform over the row)
    // Squares may have left the range of 32 bits: again with the row scaled by a power of two that brings the larger
    // of its largest |h| and sqrt(eps) to 2^31 (or as near as a normal power does), eps by its square. An
    // infinity or NaN stays as it is.
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < CH; j++) top = max(top, abs_bits8(h[j]));
    top = wave_max_u32(top);
    if constexpr (WAVES > 1) {
      __shared__ uint32_t s_top[WAVES];
      if ((t & 63) == 0) s_top[t / 64] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; w++) top = max(top, s_top[w]);
    }
    top = max(top, __float_as_uint(sqrtf(a.eps)));
    if (top < 0x7F800000u) {
      const float scale = __uint_as_float((uint32_t)min(253, 254 + 31 - (int)(top >> 23)) << 23);
#pragma unroll
      for (int j = 0; j < CH; j++) h[j] *= scale;
      mean = squares(1) / (float)a.H + a.eps * scale * scale;
    }
  }
  const float r = 1.f / sqrtf(mean);
  auto finish = [&](auto wt) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < CH; j++) {
      const int c = 8 * (j * THREADS + t), left = a.H - c;
      const f32x8 w = load_upto8<decltype(wt)::value>(a.w, c, left);
      f32x8 y;
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = h[j][i] * r * w[i];
      if (a.y) store_upto8<DT>(a.y, (size_t)row * a.ldy + c, left, y);
      if (a.q) {
        const float scale = f8_scale(row16_max_u32(abs_bits8(y)));
        if (left > 0) f8_store(a.q + (size_t)row * a.ldq + c, left, f8_pack8(y, 1.f / scale));
        if (left > 0 && (t & 15) == 0) a.scale[(size_t)row * a.lds + c / 128] = scale;
      }
    }
  };
  if (a.w_f32) finish(std::integral_constant<int, EXMOE_DTYPE_FP32>{});
  else finish(std::integral_constant<int, DT>{});
}

// ------------------------------------------------------------------------------------ host
template <int DT>
static hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  ProfScope prof("rms_norm", s);
  auto go = [&](auto waves, auto ch) {
    constexpr int WAVES = decltype(waves)::value, CH = decltype(ch)::value;
    const unsigned blocks = WAVES == 1 ? (unsigned)ceil_div(a.T, 4) : (unsigned)a.T;
    EXMOE_LAUNCH(prof, (rms_norm_kernel<DT, WAVES, CH>), dim3(blocks), dim3(WAVES == 1 ? 256 : 64 * WAVES), 0, s, a);
    return hipGetLastError();
  };
  using std::integral_constant;
  // As many waves as give each lane one chunk: a short chain of loads per row, also where rows are many (bf16
  // with residual, both outputs; one wave per row / four: 1 x 2048 5.0 / 2.7 us, 1024 x 2048 7.0 / 4.9, 4096 x
  // 2048 14.8 / 13.6; four waves / eight: 4096 x 4096 24.8 / 24.0 us, 6.3 TB/s).
  if (a.H <= 512) return go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (a.H <= 1024) return go(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  if (a.H <= 2048) return go(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (a.H <= 4096) return go(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (a.H <= 8192) return go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  return go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}

}  // namespace exmoe

using namespace exmoe;

// ------------------------------------------------------------------------------------ C ABI
extern "C" int exmoe_rms_norm(const exmoe_norm* call, hipStream_t stream) {
  EXMOE_CALL(call);
  const auto& [x, ldx, w, residual, ldr, residual_out, ldro, y, ldy, q, ldq, scale, lds, eps, T, H, dtype, w_dtype, res_dtype] = *call;
  if (T < 0) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %d)", T);
  if (T >= 1 << 22) return set_error(EXMOE_ERR_UNSUPPORTED, "T must be < 2^22 (got %d)", T);
  if (H < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "H must be positive (got %d)", H);
  if (H > kMaxDim) return set_error(EXMOE_ERR_UNSUPPORTED, "H must be <= %d (got %d)", kMaxDim, H);
  if (dtype < EXMOE_DTYPE_BF16 || dtype > EXMOE_DTYPE_FP32)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "dtype must be bf16, fp16 or fp32 (got %d)", dtype);
  if (w_dtype != dtype && w_dtype != EXMOE_DTYPE_FP32)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "w_dtype must be dtype or fp32 (got %d)", w_dtype);
  if (residual && res_dtype != dtype && res_dtype != EXMOE_DTYPE_FP32)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "res_dtype must be dtype or fp32 (got %d)", res_dtype);
  if (!(eps >= 0.f) || eps > 3.4e38f) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
  if (!y && !q) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "y and q must not both be NULL");
  if (!q != !scale) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "q and scale go together");
  if (!residual != !residual_out) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "residual and residual_out go together");
  if (T == 0) return EXMOE_OK;
  const int b = dtype_bytes(dtype), wb = dtype_bytes(w_dtype), rb = dtype_bytes(res_dtype), groups = ceil_div(H, 128);
  EXMOE_TRY(check_matrix("x", x, ldx, H, b));
  EXMOE_TRY(check_matrix("w", w, H, H, wb));
  if (y) EXMOE_TRY(check_matrix("y", y, ldy, H, b));
  if (q) EXMOE_TRY(check_matrix("q", q, ldq, H, 1));
  if (q) EXMOE_TRY(check_matrix("scale", scale, lds, groups, 4));
  if (residual) EXMOE_TRY(check_matrix("residual", residual, ldr, H, rb));
  if (residual) EXMOE_TRY(check_matrix("residual_out", residual_out, ldro, H, rb));
  const MemRows mx = mem_matrix("x", x, T, ldx, H, b), mw = mem_flat("w", w, (size_t)H * wb),
                mr = mem_matrix("residual", residual, T, ldr, H, rb), my = mem_matrix("y", y, T, ldy, H, b),
                mq = mem_matrix("q", q, T, ldq, H, 1), ms = mem_matrix("scale", scale, T, lds, groups, 4),
                mo = mem_matrix("residual_out", residual_out, T, ldro, H, rb);
  // (a row is read whole before any of it is written, so the residual may be updated in place)
  const bool in_place = residual == residual_out && (ldr == ldro || T == 1);
  if (!in_place) EXMOE_TRY(check_apart(mo, {mr}));
  EXMOE_TRY(check_apart(mo, {mx, mw}));
  EXMOE_TRY(check_apart(my, {mx, mw, mr, mo}));
  EXMOE_TRY(check_apart(mq, {mx, mw, mr, mo, my}));
  EXMOE_TRY(check_apart(ms, {mx, mw, mr, mo, my, mq}));
  NormArgs a{};
  a.x = x; a.ldx = ldx; a.w = w; a.res = residual; a.ldr = ldr; a.res_out = residual_out; a.ldro = ldro;
  a.w_f32 = w_dtype == EXMOE_DTYPE_FP32; a.res_f32 = res_dtype == EXMOE_DTYPE_FP32; a.eps = eps; a.T = T; a.H = H; a.y = y;
  a.ldy = ldy; a.q = q; a.ldq = ldq; a.scale = scale; a.lds = lds;
  return launched(by_dtype(dtype, [&](auto dt) { return launch_norm<decltype(dt)::value>(a, stream); }), "exmoe_rms_norm");
}
