// A projection shared by many requests with a low-rank adapter per request, gfx950:
//
//   y[t, :] = W x[t, :] + scale_a B_a (A_a x[t, :]),   a = adapter_ids[t]
//
// (or y[t, :] += the adapter's part when there is no W). Tokens come in any order: nothing is
// sorted. Two launches:
//   shrink  v[t, :] = A_a x[t, :] for every token with an adapter. One workgroup per 16 tokens
//           and adapter among them: the 16 tokens are one MFMA operand, so an adapter is read
//           once per 16 tokens that hold it; tokens of other adapters are computed along and
//           dropped.
//   main    the tiles of x W^T; then, per 16 tokens, one short MFMA chain per adapter among
//           them adds B_a v to the accumulators of that adapter's tokens.
// v has 32 bits but B_a v runs on 16-bit MFMA: v is scaled per token by a power of two into
// [-2, 2] and split into hi + lo, two 16-bit values whose sum is v to 2^-18 (bf16) or 2^-22
// (fp16) of it; both halves multiply the same B_a in one MFMA (16 summed positions hi, 16 lo).
// The power of two and the adapter's scale are applied in fp32 to the chain's result.
#include "exmoe.h"
#include "gemm_tile.h"

namespace exmoe {

constexpr int kMaxRank = 128;

struct LoraArgs {
  const uint16_t* x;
  const uint16_t* w;          // or null: y is read and added to
  size_t ldx, ldw, ldy;
  const uint16_t* a;          // [adapters][rank_max][K]
  const uint16_t* b;          // [adapters][N][rank_max]
  size_t lda, a_stride, ldb, b_stride;
  const int32_t* ranks;       // or null: rank_max
  const float* scales;        // or null: 1
  const int32_t* ids;
  int adapters, rank_max, T, N, K;
  uint16_t* y;
  int vec;
  uint16_t* hl;               // [T][2][rank_max]: hi and lo of the scaled v
  float* mul;                 // [T]: scale_a times the power of two taken out of v
};

__device__ __forceinline__ int token_adapter(const LoraArgs& a, int t) {
  const int id = t < a.T ? a.ids[t] : -1;
  return id >= 0 && id < a.adapters ? id : -1;
}
__device__ __forceinline__ int adapter_rank(const LoraArgs& a, int ad) {
  const int r = a.ranks ? a.ranks[ad] : a.rank_max;
  return r < 0 ? 0 : (r > a.rank_max ? a.rank_max : r);
}

// One workgroup of NW waves: 16 tokens, the j-th distinct adapter among them; the waves split
// K in 32-deep steps and their sums are added in wave order.
template <class ET, int NW>
__global__ __launch_bounds__(64 * NW) void lora_shrink_kernel(LoraArgs a) {
  constexpr int kRB = kMaxRank / 16;
  __shared__ float s_part[NW][kMaxRank][16];
  __shared__ uint32_t s_max[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t0 = blockIdx.x * 16;
  const int id = token_adapter(a, t0 + (lane & 15));
  uint32_t left = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
  int ad = -1;
  for (int j = 0; left; j++) {
    ad = __builtin_amdgcn_readlane(id, __ffs((int)left) - 1);
    if (j == (int)blockIdx.y) break;
    left &= ~(uint32_t)__ballot(id == ad);
  }
  if (!left) return;   // fewer adapters than workgroups
  if (tid < 16) s_max[tid] = 0;
  const int rank = adapter_rank(a, ad), nrb = (rank + 15) / 16;
  const int t = t0 + (lane & 15);
  const uint16_t* xp = a.x + (size_t)(t < a.T ? t : a.T - 1) * a.ldx + 8 * (lane >> 4);
  const uint16_t* ap = a.a + (size_t)ad * a.a_stride + 8 * (lane >> 4);
  f32x4 acc[kRB];
#pragma unroll
  for (int r = 0; r < kRB; r++) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
  const bf16x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k = 32 * wave; k < a.K; k += 32 * NW) {
    const bool in = k + 8 * (lane >> 4) < a.K;     // K is a multiple of 8
    const bf16x8 xv = in ? *reinterpret_cast<const bf16x8*>(xp + k) : zero;
#pragma unroll
    for (int r = 0; r < kRB; r++) {
      if (r >= nrb) break;
      const int row = 16 * r + (lane & 15);
      const bf16x8 av = in && row < rank ? *reinterpret_cast<const bf16x8*>(ap + (size_t)row * a.lda + k) : zero;
      acc[r] = ET::mfma(av, xv, acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < kRB; r++) {
    if (r >= nrb) break;
#pragma unroll
    for (int i = 0; i < 4; i++) s_part[wave][16 * r + 4 * (lane >> 4) + i][lane & 15] = acc[r][i];
  }
  __syncthreads();
  // thread: token tid % 16, rows tid / 16 + 4 NW i
  constexpr int kPer = kMaxRank / (4 * NW);
  const int tt = tid & 15, mine = t0 + tt;
  float v[kPer];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int r = (tid >> 4) + 4 * NW * i;
    v[i] = 0.f;
    if (r < rank) {
#pragma unroll
      for (int w = 0; w < NW; w++) v[i] += s_part[w][r][tt];
    }
    m = fmaxf(m, fabsf(v[i]));
  }
  atomicMax(&s_max[tt], __float_as_uint(m));   // non-negative floats order as their bits; any order, same result
  __syncthreads();
  if (mine >= a.T || token_adapter(a, mine) != ad) return;
  // 2^e with the largest |v| / 2^e in [1, 2); 1 where nothing finite and normal is there
  const uint32_t eb = s_max[tt] >> 23;
  const bool scale = eb >= 1 && eb <= 253;
  const float down = scale ? __uint_as_float((254 - eb) << 23) : 1.f, up = scale ? __uint_as_float(eb << 23) : 1.f;
  uint16_t* out = a.hl + (size_t)mine * 2 * a.rank_max;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int r = (tid >> 4) + 4 * NW * i;
    if (r < a.rank_max) {
      const float n = v[i] * down;
      const uint16_t hi = ET::from_f32(n);
      const float rest = n - ET::to_f32(hi);
      out[r] = hi;
      out[a.rank_max + r] = __builtin_isfinite(rest) ? ET::from_f32(rest) : 0;
    }
  }
  if (tid < 16) a.mul[mine] = up * (a.scales ? a.scales[ad] : 1.f);
}

// Adds the adapters' parts to the accumulators of one 16-token subtile (acc[j]: 16 columns
// n0 + 16 j..): per adapter among the tokens one chain over its rank, 16 ranks (hi and lo) a
// step, kept for the lanes of its own tokens.
template <class ET, int TQ, int STRIDE>
__device__ __forceinline__ void lora_expand(const LoraArgs& a, int t, int n0, int lane, f32x4 (&acc)[TQ][STRIDE], int i) {
  const int id = token_adapter(a, t);
  uint32_t left = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
  if (!left) return;
  const float mul = id >= 0 ? a.mul[t] : 0.f;
  const uint16_t* hl = a.hl + (size_t)(t < a.T ? t : a.T - 1) * 2 * a.rank_max + (lane >> 5) * a.rank_max;
  const bf16x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  while (left) {
    const int ad = __builtin_amdgcn_readlane(id, __ffs((int)left) - 1);
    left &= ~(uint32_t)__ballot(id == ad);
    const int rank = adapter_rank(a, ad);
    f32x4 d[TQ];
#pragma unroll
    for (int j = 0; j < TQ; j++) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < rank; r0 += 16) {
      const int col = r0 + 8 * ((lane >> 4) & 1), have = rank - col;
      const bf16x8 vv = have > 0 && id == ad ? *reinterpret_cast<const bf16x8*>(hl + col) : zero;
#pragma unroll
      for (int j = 0; j < TQ; j++) {
        int n = n0 + 16 * j + (lane & 15);
        n = n < a.N ? n : a.N - 1;
        bf16x8 bv = have > 0 ? *reinterpret_cast<const bf16x8*>(a.b + (size_t)ad * a.b_stride + (size_t)n * a.ldb + col) : zero;
        if (have < 8) {   // columns past the rank may hold anything
#pragma unroll
          for (int q = 0; q < 8; q++) bv[q] = q < have ? bv[q] : (short)0;
        }
        d[j] = ET::mfma(bv, vv, d[j]);
      }
    }
    if (id == ad) {
#pragma unroll
      for (int j = 0; j < TQ; j++)
#pragma unroll
        for (int q = 0; q < 4; q++) acc[j][i][q] += mul * d[j][q];
    }
  }
}

// One BP x BQ tile of y (BP tokens, BQ columns) per workgroup: the product with W on the
// shared tile loop (W given), the adapters' parts, one rounding.
template <class ET, int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ) void lora_tile_kernel(LoraArgs a, int p_tiles) {
  constexpr int NW = WP * WQ, TP = BP / WP / 16, TQ = BQ / WQ / 16;
  using OpP = RowOperand<BP, NW, true>;
  using OpQ = RowOperand<BQ, NW, true>;
  __shared__ __attribute__((aligned(16))) uint16_t s_p0[BP * kBK], s_p1[BP * kBK], s_q0[BQ * kBK], s_q1[BQ * kBK];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave / WQ, wq = wave % WQ;
  const int idx = xcd_contiguous(blockIdx.x, gridDim.x);
  const int p0 = idx % p_tiles * BP, q0 = idx / p_tiles * BQ;

  f32x4 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (a.w) {
    OpP op_p;
    OpQ op_q;
    op_p.init(a.x, a.K, wave, lane, [&](int i) { return (size_t)(p0 + i < a.T ? p0 + i : a.T - 1) * a.ldx; });
    op_q.init(a.w, a.K, wave, lane, [&](int i) { return (size_t)(q0 + i < a.N ? q0 + i : a.N - 1) * a.ldw; });
    const int steps = (a.K + kBK - 1) / kBK;
    auto step = [&](int s, const uint16_t* cp, const uint16_t* cq, uint16_t* np, uint16_t* nq) {
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (s + 1 < steps) {
        op_p.stage(np, (s + 1) * kBK, wave, lane);
        op_q.stage(nq, (s + 1) * kBK, wave, lane);
      }
#pragma unroll
      for (int kk = 0; kk < 2; kk++) {
        bf16x8 fq[TQ], fp[TP];
#pragma unroll
        for (int j = 0; j < TQ; j++) fq[j] = OpQ::frag(cq, (wq * TQ + j) * 16, kk, lane);
#pragma unroll
        for (int i = 0; i < TP; i++) fp[i] = OpP::frag(cp, (wp * TP + i) * 16, kk, lane);
#pragma unroll
        for (int i = 0; i < TP; i++)
#pragma unroll
          for (int j = 0; j < TQ; j++) acc[j][i] = ET::mfma(fq[j], fp[i], acc[j][i]);
      }
    };
    op_p.stage(s_p0, 0, wave, lane);
    op_q.stage(s_q0, 0, wave, lane);
    for (int s = 0; s < steps; s += 2) {
      step(s, s_p0, s_q0, s_p1, s_q1);
      if (s + 1 < steps) step(s + 1, s_p1, s_q1, s_p0, s_q0);
    }
  }

  const int n0 = q0 + wq * TQ * 16;
#pragma unroll
  for (int i = 0; i < TP; i++) {
    const int t = p0 + (wp * TP + i) * 16 + (lane & 15);
    if (!a.w && t < a.T) {
#pragma unroll
      for (int j = 0; j < TQ; j++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int n = n0 + 16 * j + 4 * (lane >> 4) + q;
          if (n < a.N) acc[j][i][q] = ET::to_f32(a.y[(size_t)t * a.ldy + n]);
        }
    }
    lora_expand<ET, TQ, TP>(a, t, n0, lane, acc, i);
    // without W, tokens without an adapter keep their y as it is
    if (t >= a.T || (!a.w && token_adapter(a, t) < 0)) continue;
#pragma unroll
    for (int j = 0; j < TQ; j++) {
      const int n = n0 + 16 * j + 4 * (lane >> 4);
      if (n < a.N) store4<ET>(a.y, (size_t)t * a.ldy + n, false, a.vec, a.N - n, acc[j][i]);
    }
  }
}

// ------------------------------------------------------------------------------------ host
static inline size_t lora_hl_bytes(int T, int rank_max) { return ((size_t)T * 2 * rank_max * 2 + 255) & ~(size_t)255; }

template <class ET>
static hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int pt = (a.T + 127) / 128, qt = (a.N + 127) / 128;
  const int distinct = a.adapters < 16 ? a.adapters : 16;
  {
    ProfScope prof("lora_shrink", s);
    EXMOE_LAUNCH(prof, (lora_shrink_kernel<ET, 4>), dim3((a.T + 15) / 16, distinct), dim3(256), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  ProfScope prof("lora_linear", s);
  EXMOE_LAUNCH(prof, (lora_tile_kernel<ET, 128, 128, 2, 2>), dim3(pt * qt), dim3(256), 0, s, a, pt);
  return hipGetLastError();
}

static int lora_shape(int T, int N, int K, int adapters, int rank_max) {
  if (T < 0 || T > (1 << 22)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "T must be in [0, 2^22] (got %d)", T);
  if (N < 1 || N > (1 << 20)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "N must be in [1, 2^20] (got %d)", N);
  if (K < 8 || K % 8 || K > (1 << 20)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "K must be a positive multiple of 8 up to 2^20 (got %d)", K);
  if (adapters < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "adapters must be positive (got %d)", adapters);
  if (rank_max < 8 || rank_max % 8 || rank_max > kMaxRank)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "rank_max must be a multiple of 8 in [8, 128] (got %d)", rank_max);
  if ((long long)((T + 127) / 128) * ((N + 127) / 128) * 256 > 0xFFFFFFFFll)
    return set_error(EXMOE_ERR_UNSUPPORTED, "T x N has too many output tiles for one launch");
  return EXMOE_OK;
}

static int check_rows16(const char* name, const void* p, size_t ld, size_t stride, int cols) {
  if (!p) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if (!aligned16(p) || ld % 8 || stride % 8)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: rows must be 16-byte aligned", name);
  if (ld < (size_t)cols) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: row stride %zu smaller than its %d columns", name, ld, cols);
  return EXMOE_OK;
}

}  // namespace exmoe

using namespace exmoe;

extern "C" size_t exmoe_lora_workspace_bytes(int T, int N, int K, int adapters, int rank_max) {
  if (lora_shape(T, N, K, adapters, rank_max)) return 0;
  return lora_hl_bytes(T, rank_max) + (size_t)T * 4;
}

extern "C" int exmoe_lora_linear(const void* x, size_t ldx, const void* w, size_t ldw, const exmoe_lora_bank* bank,
                                 const int32_t* adapter_ids, int T, int N, int K, int dtype, void* y, size_t ldy,
                                 void* workspace, size_t ws_bytes, hipStream_t stream) {
  if (!bank) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "bank must not be NULL");
  int st = lora_shape(T, N, K, bank->adapters, bank->rank_max);
  if (st) return st;
  if (dtype != EXMOE_DTYPE_BF16 && dtype != EXMOE_DTYPE_FP16)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "dtype must be bf16 or fp16 (got %d)", dtype);
  if (T == 0) return EXMOE_OK;
  if ((st = check_rows16("x", x, ldx, 0, K))) return st;
  if (w && (st = check_rows16("w", w, ldw, 0, K))) return st;
  if ((st = check_rows16("bank->a", bank->a, bank->lda, bank->a_stride, K))) return st;
  if ((st = check_rows16("bank->b", bank->b, bank->ldb, bank->b_stride, bank->rank_max))) return st;
  if (bank->adapters > 1 && (bank->a_stride < (size_t)(bank->rank_max - 1) * bank->lda + K ||
                             bank->b_stride < (size_t)(N - 1) * bank->ldb + bank->rank_max))
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "bank: adapter stride smaller than an adapter's matrix");
  if (!y || (uintptr_t)y % 2) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "y must be non-NULL and 2-byte aligned");
  if (ldy < (size_t)N) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "y: row stride %zu smaller than its %d columns", ldy, N);
  if (!adapter_ids || (uintptr_t)adapter_ids % 4 || (uintptr_t)bank->ranks % 4 || (uintptr_t)bank->scales % 4)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "adapter_ids must be non-NULL, ids, ranks and scales 4-byte aligned");
  const size_t need = exmoe_lora_workspace_bytes(T, N, K, bank->adapters, bank->rank_max);
  if (!workspace || ws_bytes < need)
    return set_error(EXMOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? ws_bytes : 0);
  if (!aligned16(workspace)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
  LoraArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.w = static_cast<const uint16_t*>(w); a.ldx = ldx; a.ldw = ldw; a.ldy = ldy;
  a.a = static_cast<const uint16_t*>(bank->a); a.b = static_cast<const uint16_t*>(bank->b); a.lda = bank->lda;
  a.a_stride = bank->a_stride; a.ldb = bank->ldb; a.b_stride = bank->b_stride; a.ranks = bank->ranks;
  a.scales = bank->scales; a.ids = adapter_ids; a.adapters = bank->adapters; a.rank_max = bank->rank_max; a.T = T;
  a.N = N; a.K = K; a.y = static_cast<uint16_t*>(y); a.vec = (uintptr_t)y % 8 == 0 && ldy % 4 == 0;
  a.hl = static_cast<uint16_t*>(workspace);
  a.mul = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + lora_hl_bytes(T, bank->rank_max));
  const hipError_t e = dtype == EXMOE_DTYPE_FP16 ? launch_lora<ElemFP16>(a, stream) : launch_lora<ElemBF16>(a, stream);
  return e == hipSuccess ? EXMOE_OK : hip_error(e, "exmoe_lora_linear");
}
