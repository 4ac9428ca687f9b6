// A projection shared by many requests with a low-rank adapter per request, gfx950:
//
//   y[t, :] = W x[t, :] + scale_a B_a (A_a x[t, :]),   a = adapter_ids[t]
//
// (or y[t, :] += the adapter's part when there is no W). Tokens come in any order: nothing is
// sorted. Two launches:
//   shrink  v[t, :] = A_a x[t, :] for every token with an adapter. One workgroup per 16 tokens,
//           adapter among them and 16 ranks of it: the 16 tokens are one MFMA operand, so an
//           adapter is read once per 16 tokens that hold it; tokens of other adapters are
//           computed along and dropped.
//   main    the tiles of x W^T; then, per 16 tokens, one short MFMA chain per adapter among
//           them adds B_a v to the accumulators of that adapter's tokens.
// v has 32 bits but B_a v runs on 16-bit MFMA: 16 ranks of a token's v are scaled by a power
// of two into [-2, 2] and split into hi + lo, two 16-bit values whose sum is v to 2^-16 (bf16)
// or 2^-22 (fp16) of it; both halves multiply the same B_a in one MFMA (16 summed positions
// hi, 16 lo). The power of two and the adapter's scale are applied in fp32 to the result.
#include "exmoe.h"
#include "gemm_wide.h"

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
  int vec8, vec16;            // rows of y can be stored 8 / 16 bytes at a time
  int rank_blocks;            // ceil(rank_max / 16)
  uint16_t* hl;               // [T][rank_blocks][2][16]: hi and lo of the scaled v
  float* mul;                 // [T][rank_blocks]: scale_a times the power of two taken out of v
};

__device__ __forceinline__ int token_adapter(const LoraArgs& a, int t) {
  const int id = t < a.T ? a.ids[t] : -1;
  return id >= 0 && id < a.adapters ? id : -1;
}
__device__ __forceinline__ int adapter_rank(const LoraArgs& a, int ad) {
  const int r = a.ranks ? a.ranks[ad] : a.rank_max;
  return r < 0 ? 0 : (r > a.rank_max ? a.rank_max : r);
}

// The j-th distinct adapter (in token order) among 16 tokens, or -1 (id: the adapter of the
// lane's token, lane % 16, or -1).
__device__ __forceinline__ int nth_adapter(int id, int j) {
  uint32_t left = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
  for (; left; j--) {
    const int ad = __builtin_amdgcn_readlane(id, __ffs((int)left) - 1);
    if (j == 0) return ad;
    left &= ~(uint32_t)__ballot(id == ad);
  }
  return -1;
}

// Workgroup (16 tokens, the j-th adapter among them, 16 ranks of it): the waves split K and
// their sums are added in wave order.
template <class ET, int NW>
__global__ __launch_bounds__(64 * NW) void lora_shrink_kernel(LoraArgs a) {
  static_assert(NW >= 4, "256 threads hold the 16 x 16 sums");
  __shared__ float s_part[NW][16][17];   // [wave][token][rank]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.x * 16, r0 = 16 * blockIdx.z;
  const int ad = nth_adapter(token_adapter(a, t0 + (lane & 15)), blockIdx.y);
  if (ad < 0) return;   // fewer adapters than workgroups
  const int rank = adapter_rank(a, ad);
  if (r0 >= rank) return;
  const int t = t0 + (lane & 15), r = r0 + (lane & 15);
  const size_t xrow[1] = {(size_t)(t < a.T ? t : a.T - 1) * a.ldx};
  const size_t arow[1] = {(size_t)ad * a.a_stride + (size_t)(r < rank ? r : rank - 1) * a.lda};
  f32x4 acc[1][1] = {{{0.f, 0.f, 0.f, 0.f}}};
  skinny_product<ET, 1, 1, NW, true>(a.x, xrow, a.a, arow, a.K, wave, lane, acc);
#pragma unroll
  for (int i = 0; i < 4; i++) s_part[wave][lane & 15][4 * (lane >> 4) + i] = acc[0][0][i];
  __syncthreads();
  // thread: token tid / 16, rank tid % 16 (rows of 16 lanes hold a token)
  const int mine = t0 + (tid >> 4);
  if (tid >= 256 || mine >= a.T || token_adapter(a, mine) != ad) return;
  float v = 0.f;
  if (r0 + (tid & 15) < rank) {
#pragma unroll
    for (int w = 0; w < NW; w++) v += s_part[w][tid >> 4][tid & 15];
  }
  float m = fabsf(v);   // (fmaxf drops a NaN)
  m = fmaxf(m, __uint_as_float(dpp_u32<0x121>(__float_as_uint(m))));
  m = fmaxf(m, __uint_as_float(dpp_u32<0x122>(__float_as_uint(m))));
  m = fmaxf(m, __uint_as_float(dpp_u32<0x124>(__float_as_uint(m))));
  m = fmaxf(m, __uint_as_float(dpp_u32<0x128>(__float_as_uint(m))));
  // 2^e with the largest |v| / 2^e in [1, 2); 1 where nothing finite and normal is there
  const uint32_t eb = __float_as_uint(m) >> 23;
  const bool scale = eb >= 1 && eb <= 253;
  const float down = scale ? __uint_as_float((254 - eb) << 23) : 1.f, up = scale ? __uint_as_float(eb << 23) : 1.f;
  const float n = v * down;
  const uint16_t hi = ET::from_f32(n);
  const float rest = n - ET::to_f32(hi);
  const size_t block = (size_t)mine * a.rank_blocks + blockIdx.z;
  uint16_t* out = a.hl + 32 * block + (tid & 15);
  out[0] = hi;
  out[16] = __builtin_isfinite(rest) ? ET::from_f32(rest) : 0;
  if ((tid & 15) == 0) a.mul[block] = up * (a.scales ? a.scales[ad] : 1.f);
}

// Eight elements of b: ranks c..c + 7 of column n, zeros from the adapter's rank on (what
// lies there may be anything).
__device__ __forceinline__ bf16x8 load_b(const LoraArgs& a, int ad, int rank, int n, int c) {
  const int have = rank - c;
  bf16x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
  if (have > 0)
    v = *reinterpret_cast<const bf16x8*>(a.b + (size_t)ad * a.b_stride + (size_t)(n < a.N ? n : a.N - 1) * a.ldb + c);
  if (have < 8) {
#pragma unroll
    for (int q = 0; q < 8; q++) v[q] = q < have ? v[q] : (short)0;
  }
  return v;
}

// Adds the adapters' parts to the sums of one block of 16 tokens and 16 columns (acc[j]:
// columns n0 + 16 j..): per adapter and 16 ranks one MFMA (hi and lo), kept for the lanes of
// the adapter's own tokens. This wave takes the adapters w, w + NW, ... among the tokens.
template <class ET, int TQ, int TP, int NW>
__device__ __forceinline__ void lora_expand16(const LoraArgs& a, int t, int n0, int wave, int lane, f32x4 (&acc)[TQ][TP],
                                              int i) {
  const int id = token_adapter(a, t);
  const size_t tok = (size_t)(t < a.T ? t : a.T - 1) * a.rank_blocks;
  uint32_t left = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
  for (int which = 0; left; which++) {
    const int ad = __builtin_amdgcn_readlane(id, __ffs((int)left) - 1);
    left &= ~(uint32_t)__ballot(id == ad);
    if (which % NW != wave) continue;
    const int rank = adapter_rank(a, ad);
    for (int rb = 0; 16 * rb < rank; rb++) {
      bf16x8 vv = {0, 0, 0, 0, 0, 0, 0, 0};
      float mul = 0.f;
      if (id == ad) {
        vv = *reinterpret_cast<const bf16x8*>(a.hl + 32 * (tok + rb) + 8 * (lane >> 4));
        mul = a.mul[tok + rb];
      }
#pragma unroll
      for (int j = 0; j < TQ; j++) {
        const f32x4 d = ET::mfma(load_b(a, ad, rank, n0 + 16 * j + (lane & 15), 16 * rb + 8 * ((lane >> 4) & 1)), vv,
                                 f32x4{0.f, 0.f, 0.f, 0.f});
        if (id == ad) {
#pragma unroll
          for (int q = 0; q < 4; q++) acc[j][i][q] += mul * d[q];
        }
      }
    }
  }
}

// The same for a block of 32 tokens and TQ blocks of 32 columns on 32 x 32 x 16 MFMA: two per
// adapter and 16 ranks (8 ranks each: hi in lanes 0..31, lo in lanes 32..63).
template <class ET, int TQ, int TP>
__device__ __forceinline__ void lora_expand32(const LoraArgs& a, int t, int n0, int lane, f32x16 (&acc)[TQ][TP], int i) {
  const int id = token_adapter(a, t);
  const size_t tok = (size_t)(t < a.T ? t : a.T - 1) * a.rank_blocks;
  uint32_t left = (uint32_t)__ballot(id >= 0);
  while (left) {
    const int ad = __builtin_amdgcn_readlane(id, __ffs((int)left) - 1);
    left &= ~(uint32_t)__ballot(id == ad);
    const int rank = adapter_rank(a, ad);
    for (int rb = 0; 16 * rb < rank; rb++) {
      bf16x8 v0 = {0, 0, 0, 0, 0, 0, 0, 0}, v1 = v0;
      float mul = 0.f;
      if (id == ad) {
        const uint16_t* p = a.hl + 32 * (tok + rb) + 16 * (lane >> 5);
        v0 = *reinterpret_cast<const bf16x8*>(p);
        v1 = *reinterpret_cast<const bf16x8*>(p + 8);
        mul = a.mul[tok + rb];
      }
#pragma unroll
      for (int j = 0; j < TQ; j++) {
        const int n = n0 + 32 * j + (lane & 31);
        f32x16 d;
#pragma unroll
        for (int q = 0; q < 16; q++) d[q] = 0.f;
        d = mfma32(ET{}, load_b(a, ad, rank, n, 16 * rb), v0, d);
        d = mfma32(ET{}, load_b(a, ad, rank, n, 16 * rb + 8), v1, d);
        if (id == ad) {
#pragma unroll
          for (int q = 0; q < 16; q++) acc[j][i][q] += mul * d[q];
        }
      }
    }
  }
}

// Few tokens: 16 TP tokens x 16 TQ columns per workgroup, W streamed once per 16 TP tokens;
// the waves split K, and the adapters among the tokens, before their sums are added.
template <class ET, int TP, int TQ, int NW>
__global__ __launch_bounds__(64 * NW) void lora_skinny_kernel(LoraArgs a) {
  __shared__ f32x4 s_part[NW][TQ * TP][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16 * TQ, t0 = blockIdx.y * 16 * TP;
  f32x4 acc[TQ][TP];
  size_t xrow[TP], wrow[TQ];
#pragma unroll
  for (int j = 0; j < TQ; j++) {
    const int n = n0 + 16 * j + (lane & 15);
    wrow[j] = (size_t)(n < a.N ? n : a.N - 1) * a.ldw;
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int i = 0; i < TP; i++) {
    const int t = t0 + 16 * i + (lane & 15);
    xrow[i] = (size_t)(t < a.T ? t : a.T - 1) * a.ldx;
  }
  if (a.w) skinny_product<ET, TP, TQ, NW, true>(a.x, xrow, a.w, wrow, a.K, wave, lane, acc);
#pragma unroll
  for (int i = 0; i < TP; i++) lora_expand16<ET, TQ, TP, NW>(a, t0 + 16 * i + (lane & 15), n0, wave, lane, acc, i);
  f32x4 v = skinny_reduce<TP, TQ, NW>(s_part, acc, wave, lane);
  const int t = t0 + 16 * (wave % TP) + (lane & 15), n = n0 + 16 * (wave / TP) + 4 * (lane >> 4);
  if (wave >= TQ * TP || t >= a.T || n >= a.N) return;
  if (!a.w) {
    if (token_adapter(a, t) < 0) return;   // keeps its y as it is
#pragma unroll
    for (int q = 0; q < 4; q++)
      if (n + q < a.N) v[q] += ET::to_f32(a.y[(size_t)t * a.ldy + n + q]);
  }
  store4<ET>(a.y, (size_t)t * a.ldy + n, false, a.vec8, a.N - n, v);
}

// Many tokens: the pipelined tiles of x W^T (gemm_wide.h), the adapters' parts added to a
// tile's sums before they are stored.
template <class ET, int TP, int TQ, int WP, int WQ, int OCC>
__global__ __launch_bounds__(64 * WP * WQ, OCC) void lora_wide_kernel(LoraArgs a, int p_tiles, int q_tiles) {
  constexpr int NW = WP * WQ, BP = 32 * TP * WP, BQ = 32 * TQ * WQ;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int pt, qt;
  band_order(xcd_contiguous(blockIdx.x, gridDim.x), p_tiles, q_tiles, pt, qt);
  const int p0 = pt * BP, q0 = qt * BQ;
  WideRows<BP, NW, 64> op_p;
  WideRows<BQ, NW, 64> op_q;
  op_p.init(make_buf(a.x, 2 * ((a.T - 1) * a.ldx + a.K)), a.K, wave, lane,
            [&](int i) { return p0 + i < a.T ? (uint32_t)((size_t)(p0 + i) * a.ldx * 2) : kNowhere; });
  op_q.init(make_buf(a.w, 2 * ((a.N - 1) * a.ldw + a.K)), a.K, wave, lane,
            [&](int i) { return q0 + i < a.N ? (uint32_t)((size_t)(q0 + i) * a.ldw * 2) : kNowhere; });
  const int n0 = q0 + 32 * TQ * (wave % WQ);
  wide_tile<ET, TP, TQ, WP, WQ, 64, false>(
      op_p, op_q, a.K, p0, a.T, q0, a.N, TileOut{a.y, 0, a.ldy, false, a.vec16 != 0}, [](int) { return 0; },
      [](int) { return 0u; }, [&](int i, int t, auto& acc) { lora_expand32<ET, TQ, TP>(a, t, n0, lane, acc, i); },
      [](int p) { return p; });
}

// ------------------------------------------------------------------------------------ host
static inline size_t lora_hl_bytes(int T, int rank_max) { return (size_t)T * ((rank_max + 15) / 16) * 64; }

template <class ET, int TP, int TQ, int NW>
static hipError_t launch_skinny(const LoraArgs& a, hipStream_t s) {
  ProfScope prof("lora_linear", s);
  EXMOE_LAUNCH(prof, (lora_skinny_kernel<ET, TP, TQ, NW>), dim3((a.N + 16 * TQ - 1) / (16 * TQ), (a.T + 16 * TP - 1) / (16 * TP)),
               dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}
template <class ET, int TP, int TQ, int WP, int WQ, int OCC>
static hipError_t launch_lora_wide(const LoraArgs& a, hipStream_t s) {
  constexpr int BP = 32 * TP * WP, BQ = 32 * TQ * WQ;
  const int pt = (a.T + BP - 1) / BP, qt = (a.N + BQ - 1) / BQ;
  ProfScope prof("lora_linear", s);
  EXMOE_LAUNCH(prof, (lora_wide_kernel<ET, TP, TQ, WP, WQ, OCC>), dim3(pt * qt), dim3(64 * WP * WQ), 0, s, a, pt, qt);
  return hipGetLastError();
}

#ifndef SKT
#define SKT 512
#endif
template <class ET>
static hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int distinct = a.adapters < 16 ? a.adapters : 16;
  {
    ProfScope prof("lora_shrink", s);
    EXMOE_LAUNCH(prof, (lora_shrink_kernel<ET, 8>), dim3((a.T + 15) / 16, distinct, a.rank_blocks), dim3(512), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool span = 2 * ((size_t)(a.T - 1) * a.ldx + a.K) < kMaxSpan && 2 * ((size_t)(a.N - 1) * a.ldw + a.K) < kMaxSpan;
  if (a.w && span && a.T > SKT) {
    if ((long long)((a.T + 255) / 256) * ((a.N + 255) / 256) >= 256) return launch_lora_wide<ET, 4, 2, 2, 4, 2>(a, s);
    return launch_lora_wide<ET, 2, 2, 2, 2, 2>(a, s);
  }
  if (a.T <= 16) return launch_skinny<ET, 1, 1, 8>(a, s);
  if (a.T <= 32) return launch_skinny<ET, 2, 1, 8>(a, s);
  return launch_skinny<ET, 4, 1, 8>(a, s);
}

static int lora_shape(int T, int N, int K, int adapters, int rank_max) {
  if (T < 0 || T > (1 << 22)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "T must be in [0, 2^22] (got %d)", T);
  if (N < 1 || N > (1 << 20)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "N must be in [1, 2^20] (got %d)", N);
  if (K < 8 || K % 8 || K > (1 << 20)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "K must be a positive multiple of 8 up to 2^20 (got %d)", K);
  if (adapters < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "adapters must be positive (got %d)", adapters);
  if (rank_max < 8 || rank_max % 8 || rank_max > kMaxRank)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "rank_max must be a multiple of 8 in [8, 128] (got %d)", rank_max);
  if ((long long)((T + 63) / 64) * ((N + 15) / 16) * 512 > 0xFFFFFFFFll)
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
  return lora_hl_bytes(T, rank_max) + (size_t)T * ((rank_max + 15) / 16) * 4;
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
  a.N = N; a.K = K; a.y = static_cast<uint16_t*>(y); a.vec8 = (uintptr_t)y % 8 == 0 && ldy % 4 == 0;
  a.vec16 = aligned16(y) && ldy % 8 == 0; a.rank_blocks = (bank->rank_max + 15) / 16;
  a.hl = static_cast<uint16_t*>(workspace);
  a.mul = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + lora_hl_bytes(T, bank->rank_max));
  const hipError_t e = dtype == EXMOE_DTYPE_FP16 ? launch_lora<ElemFP16>(a, stream) : launch_lora<ElemBF16>(a, stream);
  return e == hipSuccess ? EXMOE_OK : hip_error(e, "exmoe_lora_linear");
}
