// An expert layer in 8 bits behind its norm, of this library's own calls: the residual's addition and
// norm (16 bits for the router, 8 for the experts), routing, grouping, gate and up, silu(gate) * up with the
// routing weights in its scales, down, and the sum of each token's rows, gfx950. Of 252 us of 2048 tokens (2048
// wide, 1024 inside, 64 experts, top-8) the two products take about 195 (traced), of 100 us of 16 tokens 70.
//
// Gate and up and the down rows pass between the calls as bf16, half the bytes of fp32 and 8-bit products at full rate
// (fp32 outputs take half); the int4 layers keep both in fp32. Of the result's norm (64 tokens at these sizes,
// against 64 bits): 4.299% with bf16 rows, 4.297% with fp32 rows, 4.305% with fp32 gate and up too: the 8-bit
// activations decide. The bf16 rows alone are 0.17%, as much as the rounding of y itself. A caller who needs fp32 rows
// makes the calls one by one.
#include "checks.h"
#include "exmoe.h"
#include "fp8.h"
#include "overlap.h"
#include "row_tiles.h"

namespace exmoe {

// y[t, :] = sum_j rows[flat_to_sorted[t k + j], :] in slot order, fp32 sums of the bf16 rows, rounded once.
// One thread per 8 columns, a workgroup within one token, so that the indices of its rows are scalar loads; the
// loads of 8 rows in flight. Bound by memory (2048 tokens of 8 rows of 2048, 75 MB, 18.6 us, 4.1 TB/s: each
// workgroup's rows wait for its indices; threads numbered over all tokens' columns 22.0), for 16 tokens by the
// latency of the two loads (5 us). (Rows outside [0, n) add nothing.)
__global__ __launch_bounds__(256) void row_sum_kernel(const uint16_t* __restrict__ rows, const int32_t* __restrict__ f2s, int n,
                                                      int H, int k, uint16_t* __restrict__ y) {
  const int parts = (H / 8 + (int)blockDim.x - 1) / (int)blockDim.x, t = (int)blockIdx.x / parts;
  const int c = 8 * (((int)blockIdx.x - t * parts) * (int)blockDim.x + (int)threadIdx.x);
  if (c >= H) return;
  f32x8 sum = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int j0 = 0; j0 < k; j0 += 8) {
    f32x8 v[8];
#pragma unroll
    for (int u = 0; u < 8; u++) {
      const int s = j0 + u < k ? f2s[(size_t)t * k + j0 + u] : -1;
      v[u] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
      if (s >= 0 && s < n) v[u] = Elems<EXMOE_DTYPE_BF16>::load8(rows, (size_t)s * H + c);
    }
#pragma unroll
    for (int u = 0; u < 8; u++) sum += v[u];
  }
  Elems<EXMOE_DTYPE_BF16>::store8(y, (size_t)t * H + c, sum);
}

static inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The workspace's parts.
struct LayerFp8Parts {
  size_t x16, x8, xs, gate_up, h8, hs, rows, group, total;
  LayerFp8Parts(int T, int H, int I, int E, int k) {
    size_t at = 0;
    auto take = [&](size_t n) {
      const size_t p = at;
      at += align256(n);
      return p;
    };
    const size_t n = (size_t)T * k;
    x16 = take((size_t)T * H * 2);
    x8 = take((size_t)T * H);
    xs = take((size_t)T * (H / 128) * 4);
    gate_up = take(n * 2 * I * 2);
    h8 = take(n * I);
    hs = take(n * (I / 128) * 4);
    rows = gate_up;                       // the down rows, once gate and up are read: max(2 I, H) columns
    if ((size_t)H > 2 * (size_t)I) rows = take(n * H * 2);
    group = take(exmoe_group_workspace_bytes(T, k, E));
    total = at;
  }
};

static int check_layer(int T, int H, int I, int E, int k) {
  if (T < 0) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %d)", T);
  if (H < 1 || H % kGroup || I < 1 || I % kGroup)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "H and I must be positive multiples of 128 (got %d, %d)", H, I);
  if (E < 1 || E > kMaxExperts) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "E must be in [1, 256] (got %d)", E);
  if (k < 1 || k > E) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "k must be in [1, E] (got k=%d, E=%d)", k, E);
  if (k > kMaxK) return set_error(EXMOE_ERR_UNSUPPORTED, "k > 64 is not supported (got %d)", k);
  if (H > kMaxDim || I > kMaxDim) return set_error(EXMOE_ERR_UNSUPPORTED, "H and I must be <= %d", kMaxDim);
  // (what the product's tiles, the quantised rows and the sums hold in one launch)
  if (T >= 1 << 22 || (long long)T * k > (1 << 24) || !tiles_fit(T * k, 2 * I > H ? 2 * I : H, E, 64, 128, 256) ||
      (long long)T * k * (I / 128) > (kMaxThreads / 256) * 16 || (long long)T * (H / 8 + 255) > kMaxThreads)
    return set_error(EXMOE_ERR_UNSUPPORTED, "T*k, or T with this H, too large");
  return EXMOE_OK;
}

}  // namespace exmoe

using namespace exmoe;

// ------------------------------------------------------------------------------------ C ABI
extern "C" size_t exmoe_moe_layer_fp8_workspace_bytes(int T, int H, int I, int E, int k) {
  if (check_layer(T, H, I, E, k)) return 0;
  return LayerFp8Parts(T, H, I, E, k).total;
}

extern "C" int exmoe_moe_layer_fp8(const exmoe_layer_fp8* call, void* workspace, size_t ws_bytes, hipStream_t stream) {
  EXMOE_CALL(call);
  const exmoe_layer_fp8& c = *call;
  const int T = c.T, H = c.H, I = c.I, E = c.E, k = c.k;
  EXMOE_TRY(check_layer(T, H, I, E, k));
  if (!(c.eps >= 0.f) || c.eps > 3.4e38f) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
  const size_t n = (size_t)T * k, kh = H / 128, ki = I / 128;
  const LayerFp8Parts part(T, H, I, E, k);
  const MemRows in[] = {mem_flat("x", c.x, (size_t)T * H * 2), mem_flat("w_norm", c.w_norm, (size_t)H * 2),
                        mem_flat("w_router", c.w_router, (size_t)E * H * 2), mem_flat("gate_up", c.gate_up, (size_t)E * 2 * I * H),
                        mem_flat("gate_up_scale", c.gate_up_scale, E * 2 * ki * kh * 4), mem_flat("down", c.down, (size_t)E * H * I),
                        mem_flat("down_scale", c.down_scale, E * kh * ki * 4), mem_flat("logit_bias", c.logit_bias, (size_t)E * 4)};
  const MemRows out[] = {mem_flat("y", c.y, (size_t)T * H * 2), mem_flat("logits", c.logits, (size_t)T * E * 2),
                         mem_flat("topk_ids", c.topk_ids, n * 4), mem_flat("topk_weights", c.topk_weights, n * 4),
                         mem_flat("expert_offsets", c.expert_offsets, (size_t)(E + 1) * 4),
                         mem_flat("sorted_flat", c.sorted_flat, n * 4), mem_flat("flat_to_sorted", c.flat_to_sorted, n * 4),
                         mem_flat("residual", c.residual, (size_t)T * H * 2), mem_flat("workspace", workspace, part.total)};
  const int kIn = 8, kOut = 9;
  auto check = [&](const MemRows& m, bool may_be_null) {
    if (!m.p && !may_be_null) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must not be NULL", m.name);
    if (!aligned16(m.p)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must be 16-byte aligned", m.name);
    return (int)EXMOE_OK;
  };
  if (T == 0) {
    EXMOE_TRY(check(out[4], false));
    return exmoe_group_tokens(c.topk_ids, 0, k, E, c.expert_offsets, c.sorted_flat, c.flat_to_sorted, nullptr, 0, stream);
  }
  EXMOE_TRY(check_ws(part.total, workspace, ws_bytes));
  for (int i = 0; i < kIn; i++) EXMOE_TRY(check(in[i], i == 7));
  for (int i = 0; i < kOut; i++) {
    EXMOE_TRY(check(out[i], i == 7));
    for (const MemRows& m : in) EXMOE_TRY(check_apart(out[i], {m}));
    for (int j = 0; j < i; j++) EXMOE_TRY(check_apart(out[i], {out[j]}));
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t *x8 = ws + part.x8, *h8 = ws + part.h8;
  float *xs = reinterpret_cast<float*>(ws + part.xs), *hs = reinterpret_cast<float*>(ws + part.hs);
  uint16_t* x16 = reinterpret_cast<uint16_t*>(ws + part.x16);
  exmoe_norm nm{};
  nm.x = c.x; nm.w = c.w_norm; nm.residual = nm.residual_out = c.residual; nm.y = x16; nm.q = x8; nm.scale = xs;
  nm.ldx = nm.ldr = nm.ldro = nm.ldy = nm.ldq = H; nm.lds = kh; nm.eps = c.eps; nm.T = T; nm.H = H;
  EXMOE_TRY(exmoe_rms_norm(&nm, stream));
  EXMOE_TRY(exmoe_route_topk(x16, c.w_router, c.logit_bias, T, H, E, k, c.renormalize, c.logits, c.topk_ids, c.topk_weights, stream));
  EXMOE_TRY(exmoe_group_tokens(c.topk_ids, T, k, E, c.expert_offsets, c.sorted_flat, c.flat_to_sorted, ws + part.group,
                               exmoe_group_workspace_bytes(T, k, E), stream));
  exmoe_grouped_fp8 mm{};
  mm.x = x8; mm.ldx = H; mm.x_scale = xs; mm.ldxs = kh; mm.row_index = c.sorted_flat; mm.row_div = k; mm.x_rows = T;
  mm.expert_offsets = c.expert_offsets; mm.w = c.gate_up; mm.ldw = H; mm.w_stride = (size_t)2 * I * H; mm.w_scale = c.gate_up_scale;
  mm.ldws = kh; mm.ws_stride = 2 * ki * kh; mm.y = ws + part.gate_up; mm.ldy = 2 * I; mm.rows = (int)n; mm.N = 2 * I; mm.K = H; mm.E = E;
  mm.out_dtype = EXMOE_DTYPE_BF16;
  EXMOE_TRY(exmoe_grouped_mm_fp8(&mm, stream));
  exmoe_fp8_rows act{};
  act.x = ws + part.gate_up; act.ldx = 2 * I; act.weights = c.topk_weights; act.n_weights = (int)n; act.row_index = c.sorted_flat;
  act.q = h8; act.ldq = I; act.scale = hs; act.lds = ki; act.rows = (int)n; act.n = I; act.dtype = EXMOE_DTYPE_BF16;
  EXMOE_TRY(exmoe_swiglu_fp8(&act, stream));
  mm.x = h8; mm.ldx = I; mm.x_scale = hs; mm.ldxs = ki; mm.row_index = nullptr; mm.row_div = 1; mm.x_rows = (int)n; mm.w = c.down;
  mm.ldw = I; mm.w_stride = (size_t)H * I; mm.w_scale = c.down_scale; mm.ldws = ki; mm.ws_stride = kh * ki; mm.y = ws + part.rows;
  mm.ldy = H; mm.N = H; mm.K = I;
  EXMOE_TRY(exmoe_grouped_mm_fp8(&mm, stream));
  ProfScope prof("row_sum", stream);
  const int threads = H >= 2048 ? 256 : ceil_div(H, 512) * 64;   // (whole waves of 512 columns)
  EXMOE_LAUNCH(prof, row_sum_kernel, dim3((unsigned)(T * ceil_div(H / 8, threads))), dim3(threads), 0, stream,
               reinterpret_cast<const uint16_t*>(ws + part.rows), c.flat_to_sorted, (int)n, H, k, c.y);
  return launched(hipGetLastError(), "exmoe_moe_layer_fp8");
}
