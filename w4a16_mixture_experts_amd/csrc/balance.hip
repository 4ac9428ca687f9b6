// The losses that train a router, and their gradient, gfx950.
//
// Of the M tokens t that count (all, or those whose mask is set), with p_t = softmax(l_t) over E
// experts, lse_t = log sum_e exp(l_te), and c_e how many of their k routed ids are e:
//   balance = E sum_e f_e P_e,   f_e = c_e / (M k),   P_e = sum_t p_te / M
//   z       = sum_t lse_t^2 / M
//   d/dl_te (ga balance + gz z) = p_te / M (ga E (f_e - sum_j f_j p_tj) + 2 gz lse_t)
// (f is a count: it has no gradient). A row whose logits are all -inf has no softmax: it counts
// among the M, adds nothing to P and z, and its gradient is zero.
// Sums over tokens are made per lane (16 rows one after another, those sums in 64 bits: 2048 equal rows, as at the
// largest sizes, would be off by 2.9e-5 of their sum), then per workgroup, then over the workgroups in 64 bits, each
// in a fixed order. Bound by memory for long batches (gradient of 65536 tokens of 128 experts in 32 bits, 67 MB,
// 15 us, 4.5 TB/s) and by the latency of the two launches for short ones (8192 of 64, 1.3 MB, 5.2 and 3.0 us).
#include "checks.h"
#include "exmoe.h"
#include "fp8.h"
#include "overlap.h"
#include "row_tiles.h"

namespace exmoe {

struct BalanceArgs {
  const void* l;
  size_t ldl;
  const int32_t* ids;
  const uint8_t* mask;
  int T, E, k;
  // forward
  float* part;               // [blocks][E + 1]: sums of p, then of lse^2
  int32_t* part_n;           // [blocks][E + 1]: counts, then tokens
  float* losses;
  int32_t* counts;           // [E + 1]: c, M
  // backward
  const int32_t* counts_in;
  const float* grad;         // ga, gz
  void* dl;
  size_t lddl;
  int out_f32;
};

// Softmax of a row held by LANES neighbouring lanes, 8 experts each: v becomes exp(l - max).
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LANES >= 2) v = fmaxf(v, __uint_as_float(dpp_u32<0xB1>(__float_as_uint(v))));
  if constexpr (LANES >= 4) v = fmaxf(v, __uint_as_float(dpp_u32<0x4E>(__float_as_uint(v))));
  if constexpr (LANES >= 8) v = fmaxf(v, __uint_as_float(dpp_u32<0x141>(__float_as_uint(v))));
  if constexpr (LANES >= 16) v = fmaxf(v, __uint_as_float(dpp_u32<0x140>(__float_as_uint(v))));
  if constexpr (LANES >= 32) v = fmaxf(v, __shfl_xor(v, 16, 64));
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LANES >= 2) v += __uint_as_float(dpp_u32<0xB1>(__float_as_uint(v)));
  if constexpr (LANES >= 4) v += __uint_as_float(dpp_u32<0x4E>(__float_as_uint(v)));
  if constexpr (LANES >= 8) v += __uint_as_float(dpp_u32<0x141>(__float_as_uint(v)));
  if constexpr (LANES >= 16) v += __uint_as_float(dpp_u32<0x140>(__float_as_uint(v)));
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

constexpr float kNoLogit = -__builtin_huge_valf();

// p and lse of the row; whether it has a softmax (some logit is not -inf). A NaN or +inf among the
// logits makes them NaN, as by the formula.
template <int LANES>
__device__ __forceinline__ bool row_softmax(f32x8 l, f32x8& p, float& lse) {
  float top = l[0], s = 0.f;
#pragma unroll
  for (int i = 1; i < 8; i++) top = fmaxf(top, l[i]);
  top = lanes_max<LANES>(top);
  const bool some = !(top == kNoLogit);
  // (2^x of the rounded product x = (l - top) log2(e): off by (1 + |l - top|) 2^-24, which is small where
  // p is not)
#pragma unroll
  for (int i = 0; i < 8; i++) {
    p[i] = __builtin_amdgcn_exp2f((l[i] - (some ? top : 0.f)) * 1.4426950408889634f);
    s += p[i];
  }
  s = lanes_sum<LANES>(s);
  const bool has = some || s != s;     // (fmaxf passes over a NaN, the sum does not)
  lse = has ? (some ? top : 0.f) + logf(s) : 0.f;
  const float inv = has ? 1.f / s : 0.f;
#pragma unroll
  for (int i = 0; i < 8; i++) p[i] *= inv;
  return has;
}

// Columns of a lane (the l-th of its row's): 8 l .. 8 l + 7, or, where rows of 32 bits are read or written, 4 l .. 4 l + 3
// and as many behind the first 4 LANES, so that neighbouring lanes always touch neighbouring 16 bytes.
template <int LANES, bool SPLIT>
struct LaneCols {
  int c;
  __device__ __forceinline__ explicit LaneCols(int l) : c(SPLIT ? 4 * l : 8 * l) {}
  __device__ __forceinline__ int at(int i) const { return c + i + (SPLIT && i >= 4 ? 4 * LANES - 4 : 0); }
  template <int DT>
  __device__ __forceinline__ f32x8 load(const void* p, size_t row, int E) const {   // (past E: no logit)
    f32x8 v;
    if constexpr (SPLIT) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int c0 = at(4 * h);
        f32x4 w = {kNoLogit, kNoLogit, kNoLogit, kNoLogit};
        if (c0 + 4 <= E) {
          w = Elems<DT>::load4(p, row + c0);
        } else {
#pragma unroll
          for (int i = 0; i < 3; i++)
            if (c0 + i < E) w[i] = Elems<DT>::get(p, row + c0 + i);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) v[4 * h + i] = w[i];
      }
    } else {
      v = load_upto8<DT>(p, row + c, E - c);
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (c + i >= E) v[i] = kNoLogit;
    }
    return v;
  }
  template <int DT>
  __device__ __forceinline__ void store(void* p, size_t row, int E, f32x8 v) const {
    if constexpr (SPLIT) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int c0 = at(4 * h);
        if (c0 + 4 <= E) {
          Elems<DT>::store4(p, row + c0, f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
        } else {
#pragma unroll
          for (int i = 0; i < 3; i++)
            if (c0 + i < E) Elems<DT>::put(p, row + c0 + i, v[4 * h + i]);
        }
      }
    } else if (c < E) {
      store_upto8<DT>(p, row + c, E - c, v);
    }
  }
};

// The losses of the sums p(e) of the probabilities, z of lse^2, and the counts n(e), n(E) = M, by one wave.
template <class P, class N>
__device__ __forceinline__ void write_losses(const BalanceArgs& a, int lane, double z, P p, N n) {
  double v = 0.;
  for (int e = lane; e < a.E; e += 64) v += p(e) * (double)n(e);
  v = wave_sum(v);
  const double M = n(a.E);
  if (lane == 0) {
    a.losses[0] = M > 0. ? (float)(v * a.E / (M * M * a.k)) : 0.f;
    a.losses[1] = M > 0. ? (float)(z / M) : 0.f;
  }
}

constexpr int kFwdThreads = 1024, kBalThreads = 256;
constexpr int kRun = 16;      // rows that a lane adds up in 32 bits (64-bit sums of every row: 512 x 64 6.9 -> 7.4 us)
constexpr int kBwdRows = 4;   // rows of a lane in the backward pass, loaded together

// LANES lanes per row; a workgroup takes every gridDim.x-th run of rows, and a lone one writes the losses too.
template <int DT, int LANES>
__global__ __launch_bounds__(kFwdThreads) void balance_kernel(BalanceArgs a) {
  constexpr int kRows = kFwdThreads / LANES, kE = 8 * LANES;
  __shared__ float s_p[kFwdThreads / 64][kE + 1];
  __shared__ int s_n[kFwdThreads / 64][kE + 1];   // (a wave's own: eight experts' counters are soon contended for)
  const int t = threadIdx.x, lane = t & 63, wave = t / 64;
  const LaneCols<LANES, DT == EXMOE_DTYPE_FP32> cols(t % LANES);
  for (int e = lane; e <= kE; e += 64) s_n[wave][e] = 0;
  f32x8 sum = {0, 0, 0, 0, 0, 0, 0, 0};
  float z = 0.f;
  double long_sum[8] = {0., 0., 0., 0., 0., 0., 0., 0.}, long_z = 0.;   // of the runs before
  int n = 0, turn = 0;
  for (int r0 = blockIdx.x * kRows; r0 < a.T; r0 += gridDim.x * kRows, turn++) {
    if (turn && turn % kRun == 0) {   // (uniform)
#pragma unroll
      for (int i = 0; i < 8; i++) long_sum[i] += sum[i], sum[i] = 0.f;
      long_z += z;
      z = 0.f;
    }
    const int row = r0 + t / LANES;
    const bool live = row < a.T && (!a.mask || a.mask[row]);
    if (!live) continue;     // (the lanes of a row together)
    f32x8 p;
    float lse;
    if (row_softmax<LANES>(cols.template load<DT>(a.l, (size_t)row * a.ldl, a.E), p, lse)) {
#pragma unroll
      for (int i = 0; i < 8; i++) sum[i] += p[i];
      if (t % LANES == 0) z += lse * lse;
    }
    if (t % LANES == 0) n++;
    for (int j = t % LANES; j < a.k; j += LANES) {
      const int e = a.ids[(size_t)row * a.k + j];
      if ((unsigned)e < (unsigned)a.E) atomicAdd(&s_n[wave][e], 1);   // (whole numbers: any order)
    }
  }
  if (turn > kRun) {
#pragma unroll
    for (int i = 0; i < 8; i++) sum[i] = (float)(long_sum[i] + sum[i]);
    z = (float)(long_z + z);
  }
  // over the wave's rows, then over the waves
#pragma unroll
  for (int m = LANES; m < 64; m <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; i++) sum[i] += __shfl_xor(sum[i], m, 64);
  }
  z = wave_sum(z);
  if (lane < LANES) {
#pragma unroll
    for (int i = 0; i < 8; i++) s_p[wave][cols.at(i)] = sum[i];
  }
  if (lane == 0) s_p[wave][kE] = z;
  if (n) atomicAdd(&s_n[wave][kE], n);
  __syncthreads();
  for (int e = t; e <= a.E; e += kFwdThreads) {
    const int at = e < a.E ? e : kE;
    float v = 0.f;
    int c = 0;
#pragma unroll
    for (int w = 0; w < kFwdThreads / 64; w++) {
      v += s_p[w][at];
      c += s_n[w][at];
    }
    if (gridDim.x > 1) {
      a.part[(size_t)blockIdx.x * (a.E + 1) + e] = v;
      a.part_n[(size_t)blockIdx.x * (a.E + 1) + e] = c;
    } else {
      s_p[0][at] = v;        // (this thread alone has read the column)
      s_n[0][at] = c;
      a.counts[e] = c;
    }
  }
  if (gridDim.x > 1) return;
  __syncthreads();
  auto at = [&](int e) { return e < a.E ? e : kE; };
  if (wave == 0) write_losses(a, lane, s_p[0][kE], [&](int e) { return (double)s_p[0][at(e)]; }, [&](int e) { return s_n[0][at(e)]; });
}

// The sums over the workgroups, and the losses. 64 experts are a wave's columns, and the waves are dealt to the
// columns: those of one share its workgroups' sums and add up in wave order.
__global__ __launch_bounds__(1024) void balance_join_kernel(BalanceArgs a, int blocks) {
  constexpr int kCols = (kMaxExperts + 64) / 64 * 64;
  __shared__ double s_p[16][64];
  __shared__ int s_n[16][64];
  __shared__ double s_sum[kCols];
  __shared__ int s_cnt[kCols];
  const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
  const int chunks = a.E / 64 + 1, per = 16 / chunks, chunk = wave / per, e = 64 * chunk + lane;
  double v = 0.;
  int n = 0;
  if (chunk < chunks && e <= a.E) {
#pragma unroll 4
    for (int b = wave - chunk * per; b < blocks; b += per) {
      v += a.part[(size_t)b * (a.E + 1) + e];
      n += a.part_n[(size_t)b * (a.E + 1) + e];
    }
  }
  s_p[wave][lane] = v;
  s_n[wave][lane] = n;
  __syncthreads();
  if (chunk < chunks && wave == chunk * per) {
    for (int w = 1; w < per; w++) {
      v += s_p[wave + w][lane];
      n += s_n[wave + w][lane];
    }
    s_sum[e] = v;
    s_cnt[e] = n;
    if (e <= a.E) a.counts[e] = n;
  }
  __syncthreads();
  if (wave == 0) write_losses(a, lane, s_sum[a.E], [&](int e) { return s_sum[e]; }, [&](int e) { return s_cnt[e]; });
}

template <int DT, int LANES, bool OUT_F32>
__global__ __launch_bounds__(kBalThreads) void balance_bwd_kernel(BalanceArgs a) {
  constexpr int OT = OUT_F32 ? (int)EXMOE_DTYPE_FP32 : DT;
  constexpr int kRows = kBalThreads / LANES;   // of a workgroup at a time
  const int t = threadIdx.x;
  const LaneCols<LANES, OUT_F32 || DT == EXMOE_DTYPE_FP32> cols(t % LANES);
  const int M = a.counts_in[a.E];
  const float ga = a.grad[0] * (float)a.E, gz = 2.f * a.grad[1], per = M > 0 ? 1.f / ((float)M * (float)a.k) : 0.f,
              m = M > 0 ? 1.f / (float)M : 0.f;
  f32x8 f;
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] = cols.at(i) < a.E ? (float)a.counts_in[cols.at(i)] * per : 0.f;
  const size_t first = (size_t)blockIdx.x * kRows * kBwdRows + t / LANES;
  f32x8 l[kBwdRows];
  bool live[kBwdRows];
#pragma unroll
  for (int u = 0; u < kBwdRows; u++) {
    const size_t row = first + u * kRows;
    live[u] = M > 0 && row < (size_t)a.T && (!a.mask || a.mask[row]);
    if (live[u]) l[u] = cols.template load<DT>(a.l, row * a.ldl, a.E);
  }
#pragma unroll
  for (int u = 0; u < kBwdRows; u++) {
    const size_t row = first + u * kRows;
    f32x8 d = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live[u]) {           // (the lanes of a row together)
      f32x8 p;
      float lse;
      if (row_softmax<LANES>(l[u], p, lse)) {
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) dot += f[i] * p[i];
        dot = lanes_sum<LANES>(dot);
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] = p[i] * (ga * (f[i] - dot) + gz * lse) * m;
      }
    }
    if (row < (size_t)a.T) cols.template store<OT>(a.dl, row * a.lddl, a.E, d);
  }
}

// ------------------------------------------------------------------------------------ host
template <class F>
static hipError_t by_lanes(int E, F f) {
  if (E <= 8) return f(std::integral_constant<int, 1>{});
  if (E <= 16) return f(std::integral_constant<int, 2>{});
  if (E <= 32) return f(std::integral_constant<int, 4>{});
  if (E <= 64) return f(std::integral_constant<int, 8>{});
  if (E <= 128) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}
static int lanes_of(int E) {
  int l = 1;
  while (8 * l < E) l *= 2;
  return l;
}
// Workgroups of the forward pass: a row per LANES lanes, at most one per compute unit (what is left of the rows
// they take in turn). Large workgroups leave few sums to join (8192 tokens of 64 experts, both launches 7.5 us,
// with workgroups of 256 threads 9.4; 65536 tokens of 256 experts 25 / 40: 15 in this kernel, 10 in the join). Up to four
// runs of rows are one workgroup's, which needs no second launch (one / several and the join, replayed: 256 tokens of
// 64 experts, two runs, 5.2 / 6.7 us, 512 of 64, four, 7.0 / 6.7, 128 of 256, four, 7.6 / 7.1, 1024 of 64, eight, 10.9 /
// 6.9; a call of its own, whose second launch takes the host 3 us: 6.9 / 10.2, 7.2 / 10.2, 7.5 / 10.0).
constexpr int kLoneRuns = 4;
static int balance_blocks(int T, int E) {
  const long long n = ((long long)T * lanes_of(E) + kFwdThreads - 1) / kFwdThreads;
  return n > 256 ? 256 : (n <= kLoneRuns ? 1 : (int)n);
}

}  // namespace exmoe

using namespace exmoe;

// ------------------------------------------------------------------------------------ C ABI
static int check_router(int T, int E, int k, int dtype) {
  if (T < 0 || T > (1 << 24)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "T must be in [0, 2^24] (got %d)", T);
  if (E < 1 || E > kMaxExperts) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "E must be in [1, 256] (got %d)", E);
  if (k < 1 || k > E) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "k must be in [1, E] (got k=%d, E=%d)", k, E);
  if (k > kMaxK) return set_error(EXMOE_ERR_UNSUPPORTED, "k > 64 is not supported (got %d)", k);
  if (dtype < EXMOE_DTYPE_BF16 || dtype > EXMOE_DTYPE_FP32)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "dtype must be bf16, fp16 or fp32 (got %d)", dtype);
  return EXMOE_OK;
}

extern "C" size_t exmoe_balance_loss_workspace_bytes(int T, int E) {
  if (check_router(T, E, 1, EXMOE_DTYPE_BF16)) return 0;
  return (size_t)balance_blocks(T, E) * (E + 1) * 8;
}

extern "C" int exmoe_balance_loss(const exmoe_balance* call, void* workspace, size_t ws_bytes, hipStream_t stream) {
  EXMOE_CALL(call);
  const void* logits = call->logits;
  const int32_t* topk_ids = call->topk_ids;
  const uint8_t* mask = call->mask;
  float* losses = call->losses;
  int32_t* counts = call->counts;
  const size_t ldl = call->ldl;
  const int T = call->T, E = call->E, k = call->k, dtype = call->dtype;
  EXMOE_TRY(check_router(T, E, k, dtype));
  if (!losses || (uintptr_t)losses % 4) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "losses must be non-NULL and 4-byte aligned");
  EXMOE_TRY(check_int32("counts", counts, false));
  const int b = dtype_bytes(dtype);
  if (T > 0) {
    EXMOE_TRY(check_matrix("logits", logits, ldl, E, b));
    EXMOE_TRY(check_int32("topk_ids", topk_ids, false));
  }
  const size_t need = exmoe_balance_loss_workspace_bytes(T, E);
  EXMOE_TRY(check_ws(need, workspace, ws_bytes));
  const MemRows ml = mem_matrix("logits", logits, T, ldl, E, b), mi = mem_flat("topk_ids", topk_ids, (size_t)T * k * 4),
                mm = mem_flat("mask", mask, T), mo = mem_flat("losses", losses, 8), mc = mem_flat("counts", counts, (E + 1) * 4);
  EXMOE_TRY(check_apart(mo, {ml, mi, mm, mc}));
  EXMOE_TRY(check_apart(mc, {ml, mi, mm}));
  EXMOE_TRY(check_apart(mem_flat("workspace", workspace, need), {ml, mi, mm, mo, mc}));
  BalanceArgs a{};
  a.l = logits; a.ldl = ldl; a.ids = topk_ids; a.mask = mask; a.T = T; a.E = E; a.k = k; a.losses = losses; a.counts = counts;
  const int blocks = balance_blocks(T, E);
  a.part = static_cast<float*>(workspace);
  a.part_n = reinterpret_cast<int32_t*>(a.part + (size_t)blocks * (E + 1));
  return launched(by_dtype(dtype, [&](auto dt) {
                    return by_lanes(E, [&](auto lanes) {
                      ProfScope prof("balance_loss", stream);
                      EXMOE_LAUNCH(prof, (balance_kernel<decltype(dt)::value, decltype(lanes)::value>), dim3(blocks),
                                   dim3(kFwdThreads), 0, stream, a);
                      const hipError_t e = hipGetLastError();
                      if (e != hipSuccess || blocks == 1) return e;
                      ProfScope join("balance_join", stream);
                      EXMOE_LAUNCH(join, balance_join_kernel, dim3(1), dim3(1024), 0, stream, a, blocks);
                      return hipGetLastError();
                    });
                  }),
                  "exmoe_balance_loss");
}

extern "C" int exmoe_balance_loss_backward(const exmoe_balance* call, hipStream_t stream) {
  EXMOE_CALL(call);
  const void* logits = call->logits;
  const int32_t* counts = call->counts;
  const uint8_t* mask = call->mask;
  const float* grad_losses = call->grad_losses;
  void* dlogits = call->dlogits;
  const size_t ldl = call->ldl, lddl = call->lddl;
  const int T = call->T, E = call->E, k = call->k, dtype = call->dtype, out_dtype = call->out_dtype;
  EXMOE_TRY(check_router(T, E, k, dtype));
  if (out_dtype != dtype && out_dtype != EXMOE_DTYPE_FP32)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "out_dtype must be dtype or fp32 (got %d)", out_dtype);
  if (T == 0) return EXMOE_OK;
  const int b = dtype_bytes(dtype), ob = dtype_bytes(out_dtype);
  EXMOE_TRY(check_matrix("logits", logits, ldl, E, b));
  EXMOE_TRY(check_int32("counts", counts, false));
  if (!grad_losses || (uintptr_t)grad_losses % 4)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "grad_losses must be non-NULL and 4-byte aligned");
  EXMOE_TRY(check_matrix("dlogits", dlogits, lddl, E, ob));
  // (a row is read whole before it is written: dlogits may lie on logits of its type)
  const bool in_place = dlogits == logits && b == ob && (ldl == lddl || T == 1);
  const MemRows ml = mem_matrix("logits", logits, T, ldl, E, b), mc = mem_flat("counts", counts, (E + 1) * 4),
                mm = mem_flat("mask", mask, T), mg = mem_flat("grad_losses", grad_losses, 8),
                md = mem_matrix("dlogits", dlogits, T, lddl, E, ob);
  if (!in_place) EXMOE_TRY(check_apart(md, {ml}));
  EXMOE_TRY(check_apart(md, {mc, mm, mg}));
  BalanceArgs a{};
  a.l = logits; a.ldl = ldl; a.mask = mask; a.T = T; a.E = E; a.k = k; a.counts_in = counts; a.grad = grad_losses;
  a.dl = dlogits; a.lddl = lddl; a.out_f32 = ob == 4;
  return launched(by_dtype(dtype, [&](auto dt) {
                    return by_lanes(E, [&](auto lanes) {
                      constexpr int DT = decltype(dt)::value, LANES = decltype(lanes)::value;
                      const unsigned blocks = (unsigned)(((size_t)T * LANES + kBalThreads * kBwdRows - 1) / (kBalThreads * kBwdRows));
                      ProfScope prof("balance_loss_bwd", stream);
                      if (a.out_f32)
                        EXMOE_LAUNCH(prof, (balance_bwd_kernel<DT, LANES, true>), dim3(blocks), dim3(kBalThreads), 0, stream, a);
                      else
                        EXMOE_LAUNCH(prof, (balance_bwd_kernel<DT, LANES, false>), dim3(blocks), dim3(kBalThreads), 0, stream, a);
                      return hipGetLastError();
                    });
                  }),
                  "exmoe_balance_loss_backward");
}
