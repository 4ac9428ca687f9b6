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
// of two and split into four 16-bit terms (SplitV); two of them multiply the same B_a in one
// MFMA of 32 summed positions (16 ranks each), the other two in a second one. The power of two
// and the adapter's scale are applied in fp32 to the result. (Two terms alone are off by 2^-16
// of v in bf16 and lose ranks far below the token's largest in fp16. The second MFMA and its
// operand cost: 2048 tokens of 8 requests, rank 64, 4096 x 4096, 80.0 -> 82.6 us for the main
// launch; 64 tokens of 64 requests, 2048 x 2048, 9.9 -> 10.6; one token, rank 16, 5.4 -> 5.5.)
#include <algorithm>

#include "exmoe.h"
#include "gemm_wide.h"
#include "overlap.h"

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
  // by groups of 16 tokens and blocks of 16 ranks (group g, block b: index g rank_blocks + b):
  uint16_t* terms;            // [index][4][2][16][8]: term; ranks 0..7, 8..15; token; rank (fragment order)
  float* mul;                 // [index][16]: scale_a times the power of two taken out of a token's v
  int2* info;                 // [T]: the token's adapter (-1: none) and its rank
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

// A token's v of 16 ranks as four 16-bit terms: m, the largest |v| of the 16, is scaled into
// [2^kTop, 2^(kTop + 1)), and v down = t0 + t1 + (t2 + t3) / kRest, each term what the ones before
// leave, rounded to nearest (every difference is exact).
//   bf16: three terms hold the 24 bits, in fp32's own range of exponents: nothing is lost.
//   fp16: t0 + t1 are off by 2^-22 of the value or, where t1 is subnormal, by 2^-25; t2 and t3 take
//   that 2^23 times larger (at most 2^15) and are off by 2^-25 of it. Nothing is lost of ranks down
//   to 2^-38 of the largest, below that at most 2^-62 of the largest.
template <class ET>
struct SplitV {
  static constexpr bool kBF16 = std::is_same_v<ET, ElemBF16>;
  static constexpr uint32_t kTop = kBF16 ? 0 : 14;
  static constexpr float kRest = kBF16 ? 1.f : 8388608.f;
  float down, up;   // the power of two and its inverse; 1 where nothing finite and normal is there
  __device__ __forceinline__ explicit SplitV(float m) {
    const uint32_t eb = __float_as_uint(m) >> 23;
    const bool scale = eb > kTop && eb <= (kBF16 ? 253 : 254);
    down = scale ? __uint_as_float((254 + kTop - eb) << 23) : 1.f;
    up = scale ? __uint_as_float((eb - kTop) << 23) : 1.f;
  }
  // term i to out[256 i]
  __device__ __forceinline__ void split(float v, uint16_t* out) const {
    float r = v * down;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint16_t t = kBF16 && i == 3 ? 0 : ET::from_f32(r);   // (after three bf16 terms nothing is left)
      out[256 * i] = t;
      r -= ET::to_f32(t);
      if (i == 0 && !__builtin_isfinite(r)) r = 0.f;   // (an infinite or NaN v: the first term has it)
      if (i == 1) r *= kRest;
    }
  }
};

// B v of 16 ranks: v0 holds the terms 0 and 1, v1 the terms 2 and 3.
template <class ET>
__device__ __forceinline__ f32x4 times_v(bf16x8 b, bf16x8 v0, bf16x8 v1) {
  f32x4 d = ET::mfma(b, v1, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
  for (int q = 0; q < 4; q++) d[q] *= 1.f / SplitV<ET>::kRest;
  return ET::mfma(b, v0, d);
}

// Workgroup (16 tokens, the y-th adapter among them and every gridDim.y-th after it, 16
// ranks): the waves split K and their sums are added in wave order.
template <class ET, int NW, int D>
__global__ __launch_bounds__(64 * NW) void lora_shrink_kernel(LoraArgs a) {
  static_assert(NW >= 4, "256 threads hold the 16 x 16 sums");
  __shared__ __attribute__((aligned(16))) uint16_t s_a[NW][32 * D], s_b[NW][32 * D];
  __shared__ float s_part[NW][16][17];   // [wave][token][rank]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.x * 16, r0 = 16 * blockIdx.z, t = t0 + (lane & 15);
  const int id = token_adapter(a, t), mine = t0 + ((tid >> 4) & 15), mine_id = token_adapter(a, mine);
  if (blockIdx.y == 0 && blockIdx.z == 0 && tid < 16 && t < a.T) a.info[t] = make_int2(id, id >= 0 ? adapter_rank(a, id) : 0);
  NarrowRows<16, D> op_x, op_a;
  op_x.init(make_buf(a.x + (size_t)t0 * a.ldx, 2 * ((size_t)(min(16, a.T - t0) - 1) * a.ldx + a.K)), a.K, lane,
            [&](int i) { return t0 + i < a.T ? (uint32_t)(i * a.ldx * 2) : kNowhere; });
  for (int j = blockIdx.y;; j += gridDim.y) {
    const int ad = nth_adapter(id, j);
    if (ad < 0) return;   // fewer adapters than workgroups
    const int rank = adapter_rank(a, ad);
    if (r0 >= rank) continue;
    op_a.init(make_buf(a.a + (size_t)ad * a.a_stride + (size_t)r0 * a.lda, 2 * ((size_t)(min(16, rank - r0) - 1) * a.lda + a.K)),
              a.K, lane, [&](int i) { return r0 + i < rank ? (uint32_t)(i * a.lda * 2) : kNowhere; });
    f32x4 acc[1][1] = {{{0.f, 0.f, 0.f, 0.f}}};
    narrow_product<ET, 1, 1, NW, D>(op_x, op_a, a.K, wave, lane, s_a[wave], s_b[wave], acc);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; i++) s_part[wave][lane & 15][4 * (lane >> 4) + i] = acc[0][0][i];
    __syncthreads();
    // thread: token tid / 16, rank tid % 16 (rows of 16 lanes hold a token)
    if (tid >= 256 || mine_id != ad) continue;
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
    const SplitV<ET> sv(m);
    const size_t block = (size_t)blockIdx.x * a.rank_blocks + blockIdx.z;
    sv.split(v, a.terms + 1024 * block + 128 * ((tid >> 3) & 1) + 8 * (tid >> 4) + (tid & 7));
    if ((tid & 15) == 0) a.mul[16 * block + (tid >> 4)] = sv.up * (a.scales ? a.scales[ad] : 1.f);
  }
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

// The adapters' parts of one block of 16 tokens and 16 columns from n0 that this wave adds:
// those of the adapters wave + m NW (m < kSlots) among the tokens, in token order. The first
// 64 ranks of their B are loaded when they are found, ahead of the pass over K; add() runs
// two MFMAs (the terms of v) per adapter and 16 ranks, kept for the lanes of the adapter's own tokens.
template <class ET, int NW>
struct ExpandBlock {
  static constexpr int kSlots = 16 / NW;
  int id;
  size_t group;              // first block index of the 16 tokens
  int ad[kSlots], rank[kSlots];
  bf16x8 bv[kSlots][4];

  __device__ __forceinline__ void find(const LoraArgs& a, int t0, int2 info, int n0, int wave, int lane) {
    id = info.x;
    group = (size_t)min(t0 / 16, (a.T - 1) / 16) * a.rank_blocks;
    uint32_t left = (uint32_t)__ballot(info.y > 0) & 0xFFFFu;
    int which = 0;
#pragma unroll
    for (int m = 0; m < kSlots; m++) {
      ad[m] = 0;
      rank[m] = 0;
      for (bool found = false; left && !found; which++) {
        const int lead = __ffs((int)left) - 1, cand = __builtin_amdgcn_readlane(id, lead);
        left &= ~(uint32_t)__ballot(id == cand);
        found = which == wave + m * NW;
        if (found) {
          ad[m] = cand;
          rank[m] = __builtin_amdgcn_readlane(info.y, lead);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; u++)
        bv[m][u] = load_b(a, ad[m], rank[m], n0 + (lane & 15), 16 * u + 8 * ((lane >> 4) & 1));
    }
  }
  __device__ __forceinline__ void add(const LoraArgs& a, int n0, int lane, f32x4& acc) {
#pragma unroll
    for (int m = 0; m < kSlots; m++) {
      for (int r0 = 0; r0 < rank[m]; r0 += 64) {
        bf16x8 v0[4], v1[4];
        float mul[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const size_t blk = group + (r0 + 16 * u < rank[m] ? r0 / 16 + u : 0);
          v0[u] = *reinterpret_cast<const bf16x8*>(a.terms + 1024 * blk + 8 * lane);   // (tokens of other adapters: dropped)
          v1[u] = *reinterpret_cast<const bf16x8*>(a.terms + 1024 * blk + 512 + 8 * lane);
          mul[u] = a.mul[16 * blk + (lane & 15)];
          if (r0) bv[m][u] = load_b(a, ad[m], rank[m], n0 + (lane & 15), r0 + 16 * u + 8 * ((lane >> 4) & 1));
        }
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const f32x4 d = times_v<ET>(bv[m][u], v0[u], v1[u]);
          if (id == ad[m] && r0 + 16 * u < rank[m]) {
#pragma unroll
            for (int q = 0; q < 4; q++) acc[q] += mul[u] * d[q];
          }
        }
      }
    }
  }
};

// The same by one wave for TQ blocks of 16 columns: kBatch (adapter, 16 ranks) pairs at a time,
// whose loads run together; the first of them are issued before the pass over W.
template <class ET, int TQ>
struct ExpandWave {
  static constexpr int kBatch = 4;
  int id, y;
  size_t group;
  uint32_t left;
  int ad, rank, next;        // the walk: ranks from `next` on of adapter `ad`
  int got[kBatch];           // adapter of each pair, or -1
  bf16x8 bv[kBatch][TQ], v0[kBatch], v1[kBatch];
  float mul[kBatch];

  __device__ __forceinline__ void start(const LoraArgs& a, int t0, int lane) {
    const int t = t0 + (lane & 15);
    const int2 info = t < a.T ? a.info[t] : make_int2(-1, 0);
    id = info.x;
    y = info.y;
    group = (size_t)min(t0 / 16, (a.T - 1) / 16) * a.rank_blocks;
    left = (uint32_t)__ballot(info.y > 0) & 0xFFFFu;
    ad = rank = next = 0;
  }
  __device__ __forceinline__ void load(const LoraArgs& a, int n0, int lane) {
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      if (next >= rank && left) {
        const int lead = __ffs((int)left) - 1;
        ad = __builtin_amdgcn_readlane(id, lead);
        rank = __builtin_amdgcn_readlane(y, lead);
        left &= ~(uint32_t)__ballot(id == ad);
        next = 0;
      }
      const bool have = next < rank;
      got[u] = have ? ad : -1;
      const size_t blk = group + (have ? next / 16 : 0);
#pragma unroll
      for (int j = 0; j < TQ; j++)
        bv[u][j] = load_b(a, have ? ad : 0, have ? rank : 0, n0 + 16 * j + (lane & 15), next + 8 * ((lane >> 4) & 1));
      v0[u] = *reinterpret_cast<const bf16x8*>(a.terms + 1024 * blk + 8 * lane);   // (tokens of other adapters: dropped)
      v1[u] = *reinterpret_cast<const bf16x8*>(a.terms + 1024 * blk + 512 + 8 * lane);
      mul[u] = a.mul[16 * blk + (lane & 15)];
      next += 16;
    }
  }
  __device__ __forceinline__ bool more() const { return left || next < rank; }
  __device__ __forceinline__ void add(f32x4 (&acc)[TQ]) {
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
#pragma unroll
      for (int j = 0; j < TQ; j++) {
        const f32x4 d = times_v<ET>(bv[u][j], v0[u], v1[u]);
        if (got[u] >= 0 && id == got[u]) {
#pragma unroll
          for (int q = 0; q < 4; q++) acc[j][q] += mul[u] * d[q];
        }
      }
    }
  }
};

// The same for a block of 32 tokens and TQ blocks of 32 columns on 32 x 32 x 16 MFMA: four per
// adapter and 16 ranks (8 ranks and two terms of v each, one in lanes 0..31, one in 32..63).
template <class ET, int TQ, int TP>
__device__ __forceinline__ void lora_expand32(const LoraArgs& a, int t, int n0, int lane, f32x16 (&acc)[TQ][TP], int i) {
  const int2 info = t < a.T ? a.info[t] : make_int2(-1, 0);
  const int id = info.x;
  const size_t group = (size_t)((t < a.T ? t : a.T - 1) / 16) * a.rank_blocks;
  uint32_t left = (uint32_t)__ballot(id >= 0);
  while (left) {
    const int lead = __ffs((int)left) - 1;
    const int ad = __builtin_amdgcn_readlane(id, lead), rank = __builtin_amdgcn_readlane(info.y, lead);
    left &= ~(uint32_t)__ballot(id == ad);
    // two blocks of 16 ranks a turn, their loads together
    for (int rb = 0; 16 * rb < rank; rb += 2) {
      bf16x8 v[2][2][2], bv[2][TQ][2];   // v: [16 ranks][terms 0, 1 or 2, 3][8 ranks]
      float mul[2];
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const bool in = 16 * (rb + u) < rank;
        const size_t blk = group + (in ? rb + u : 0);
        const uint16_t* p = a.terms + 1024 * blk + 256 * (lane >> 5) + 8 * (lane & 15);
#pragma unroll
        for (int m = 0; m < 2; m++)
#pragma unroll
          for (int h = 0; h < 2; h++) v[u][m][h] = *reinterpret_cast<const bf16x8*>(p + 512 * m + 128 * h);   // (tokens of other adapters: dropped)
        mul[u] = a.mul[16 * blk + (lane & 15)];
#pragma unroll
        for (int j = 0; j < TQ; j++)
#pragma unroll
          for (int h = 0; h < 2; h++) bv[u][j][h] = load_b(a, ad, rank, n0 + 32 * j + (lane & 31), 16 * (rb + u) + 8 * h);
      }
#pragma unroll
      for (int u = 0; u < 2; u++) {
        if (16 * (rb + u) >= rank) break;
#pragma unroll
        for (int j = 0; j < TQ; j++) {
          f32x16 d;
#pragma unroll
          for (int q = 0; q < 16; q++) d[q] = 0.f;
          d = mfma32(ET{}, bv[u][j][0], v[u][1][0], d);
          d = mfma32(ET{}, bv[u][j][1], v[u][1][1], d);
#pragma unroll
          for (int q = 0; q < 16; q++) d[q] *= 1.f / SplitV<ET>::kRest;
          d = mfma32(ET{}, bv[u][j][0], v[u][0][0], d);
          d = mfma32(ET{}, bv[u][j][1], v[u][0][1], d);
          if (id == ad) {
#pragma unroll
            for (int q = 0; q < 16; q++) acc[j][i][q] += mul[u] * d[q];
          }
        }
      }
    }
  }
}

// Columns n..n + 3 of token t: the sums, rounded, or added to y when there is no W.
template <class ET>
__device__ __forceinline__ void lora_store(const LoraArgs& a, int t, int n, f32x4 v) {
  if (t >= a.T || n >= a.N) return;
  if (!a.w) {
    if (token_adapter(a, t) < 0) return;   // keeps its y as it is
#pragma unroll
    for (int q = 0; q < 4; q++)
      if (n + q < a.N) v[q] += ET::to_f32(a.y[(size_t)t * a.ldy + n + q]);
  }
  store4<ET>(a.y, (size_t)t * a.ldy + n, false, a.vec8, a.N - n, v);
}

// Few tokens: 16 tokens x 16 columns per workgroup, W streamed once per 16 tokens; the waves
// split K, and the adapters among the tokens, before their sums are added.
template <class ET, int NW, int D>
__global__ __launch_bounds__(64 * NW) void lora_skinny_kernel(LoraArgs a) {
  constexpr int kPart = 32 * D;
  __shared__ __attribute__((aligned(16))) uint16_t s_a[NW][kPart], s_b[NW][kPart];
  static_assert(sizeof(f32x4) * 64 <= sizeof(s_a[0]), "the sums fit into the slices' part");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 16, t = t0 + (lane & 15);
  f32x4 acc[1][1] = {{{0.f, 0.f, 0.f, 0.f}}};
  ExpandBlock<ET, NW> part;
  part.find(a, t0, t < a.T ? a.info[t] : make_int2(-1, 0), n0, wave, lane);
  if (a.w) {
    NarrowRows<16, D> op_x, op_w;
    op_x.init(make_buf(a.x + (size_t)t0 * a.ldx, 2 * ((size_t)(min(16, a.T - t0) - 1) * a.ldx + a.K)), a.K, lane,
              [&](int i) { return t0 + i < a.T ? (uint32_t)(i * a.ldx * 2) : kNowhere; });
    op_w.init(make_buf(a.w + (size_t)n0 * a.ldw, 2 * ((size_t)(min(16, a.N - n0) - 1) * a.ldw + a.K)), a.K, lane,
              [&](int i) { return n0 + i < a.N ? (uint32_t)(i * a.ldw * 2) : kNowhere; });
    narrow_product<ET, 1, 1, NW, D>(op_x, op_w, a.K, wave, lane, s_a[wave], s_b[wave], acc);
  }
  part.add(a, n0, lane, acc[0][0]);
  __syncthreads();
  f32x4 v[1];
  skinny_reduce<1, 1, NW>(reinterpret_cast<f32x4(*)[1][64]>(&s_a[0][0]), acc, wave, lane, v);
  if (wave == 0) lora_store<ET>(a, t, n0 + 4 * (lane >> 4), v[0]);
}

// More tokens, still too few for the pipelined tiles: 16 TP tokens x 16 TQ columns per workgroup,
// the waves split K; a wave adds the adapters of the 16 tokens whose sums it joins.
template <class ET, int TP, int TQ>
__global__ __launch_bounds__(256) void lora_mid_kernel(LoraArgs a, int t_tiles) {
  constexpr int NW = 4, D = 64, kPart = 16 * (TP + TQ) * D;
  __shared__ __attribute__((aligned(16))) uint16_t s_a[2][NW][kPart];   // two slices a wave
  static_assert(sizeof(f32x4) * TP * TQ * 64 * NW <= sizeof(s_a), "the sums fit into the slices' part");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // (the blocks of one column block on one XCD: W is read into one L2)
  const int idx = xcd_contiguous(blockIdx.x, gridDim.x);
  const int n0 = idx / t_tiles * 16 * TQ, t0 = idx % t_tiles * 16 * TP;
  ExpandWave<ET, TQ> part;   // (of the 16 tokens whose sums this wave joins)
  static_assert(TP <= NW, "a wave per 16 tokens");
  if (wave < TP) {
    part.start(a, t0 + 16 * wave, lane);
    part.load(a, n0, lane);
  }
  f32x4 acc[TQ][TP];
#pragma unroll
  for (int i = 0; i < TP; i++)
#pragma unroll
    for (int j = 0; j < TQ; j++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (a.w) {
    NarrowRows<16 * TP, D> op_x;
    NarrowRows<16 * TQ, D> op_w;
    op_x.init(make_buf(a.x + (size_t)t0 * a.ldx, 2 * ((size_t)(min(16 * TP, a.T - t0) - 1) * a.ldx + a.K)), a.K, lane,
              [&](int i) { return t0 + i < a.T ? (uint32_t)(i * a.ldx * 2) : kNowhere; });
    op_w.init(make_buf(a.w + (size_t)n0 * a.ldw, 2 * ((size_t)(min(16 * TQ, a.N - n0) - 1) * a.ldw + a.K)), a.K, lane,
              [&](int i) { return n0 + i < a.N ? (uint32_t)(i * a.ldw * 2) : kNowhere; });
    narrow_product<ET, TP, TQ, NW, D>(op_x, op_w, a.K, wave, lane, s_a[0][wave], s_a[1][wave], acc);
  }
  __syncthreads();
  f32x4 v[TQ];
  skinny_reduce<TP, TQ, NW>(reinterpret_cast<f32x4(*)[TQ * TP][64]>(&s_a[0][0][0]), acc, wave, lane, v);
  if (wave >= TP) return;
  part.add(v);
  while (part.more()) {
    part.load(a, n0, lane);
    part.add(v);
  }
#pragma unroll
  for (int j = 0; j < TQ; j++) lora_store<ET>(a, t0 + 16 * wave + (lane & 15), n0 + 16 * j + 4 * (lane >> 4), v[j]);
}

// One to sixteen tokens with few 16-rank blocks among their adapters (at most NB): both
// products in one launch. Every workgroup makes v for itself, from A blocks that ride along
// the pass over K as further column blocks of the product (A_a is read by every workgroup,
// from the caches); the adapter's B blocks are loaded behind it.
template <class ET, int NB, int NW>
__global__ __launch_bounds__(64 * NW) void lora_token_kernel(LoraArgs a) {
  constexpr int D = 64, kPart = 16 * (2 + NB) * D, kCopies = 2 * (2 + NB);
  __shared__ __attribute__((aligned(16))) uint16_t s_a[NW][kPart], s_b[NW][kPart];
  static_assert(sizeof(f32x4) * (1 + NB) * 64 <= sizeof(s_a[0]), "the sums fit into the slices' part");
  __shared__ __attribute__((aligned(16))) uint16_t s_terms[NB][1024];
  __shared__ float s_mul[NB][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16, t = lane & 15, n = n0 + (lane & 15);
  // the first slices of x and W are on their way while the adapters are found; ranks come by
  // scalar loads (constant address space), which do not wait for them
  const int id = token_adapter(a, t);
  NarrowRows<16, D> op_x, op_w, op_a[NB];
  op_x.init(make_buf(a.x, 2 * ((size_t)(a.T - 1) * a.ldx + a.K)), a.K, lane,
            [&](int i) { return i < a.T ? (uint32_t)(i * a.ldx * 2) : kNowhere; });
  // (without W every copy of it moves nothing: its rows are zeros)
  op_w.init(make_buf(a.w ? a.w + (size_t)n0 * a.ldw : a.x, a.w ? 2 * ((size_t)(min(16, a.N - n0) - 1) * a.ldw + a.K) : 0),
            a.w ? a.K : 0, lane, [&](int i) { return a.w && n0 + i < a.N ? (uint32_t)(i * a.ldw * 2) : kNowhere; });
  uint16_t *const la = s_a[wave], *const lb = s_b[wave];
  auto issue_xw = [&](int s, uint16_t* lds) __attribute__((always_inline)) {
    const int k0 = (s * NW + wave) * D;
    op_x.stage(lds, k0);
    op_w.stage(lds + 16 * D, k0);
  };
  issue_xw(0, la);
  issue_xw(1, lb);
  const auto* ranks = (const __attribute__((address_space(4))) int32_t*)a.ranks;
  // block b: 16 ranks from bfirst[b] on of adapter bad[b], of rank brank[b] (0: no block)
  int bad[NB], bfirst[NB], brank[NB];
  {
    uint32_t left = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
    int ad = 0, rank = 0, next = 0;
#pragma unroll
    for (int b = 0; b < NB; b++) {
      if (next >= rank) {
        rank = 0;
        while (left && rank <= 0) {   // (an adapter of rank 0 has no block)
          ad = __builtin_amdgcn_readlane(id, __ffs((int)left) - 1);
          rank = a.ranks ? min(ranks[ad], a.rank_max) : a.rank_max;
          left &= ~(uint32_t)__ballot(id == ad);
        }
        rank = max(rank, 0);
        next = 0;
      }
      bad[b] = ad;
      bfirst[b] = next;
      brank[b] = rank;
      next += 16;
    }
  }
#pragma unroll
  for (int b = 0; b < NB; b++) {
    const int rows = min(16, brank[b] - bfirst[b]);
    op_a[b].init(make_buf(a.a + (size_t)bad[b] * a.a_stride + (size_t)bfirst[b] * a.lda,
                          rows > 0 ? 2 * ((size_t)(rows - 1) * a.lda + a.K) : 0),
                 rows > 0 ? a.K : 0, lane, [&](int i) { return i < rows ? (uint32_t)(i * a.lda * 2) : kNowhere; });
  }
  auto issue_a = [&](int s, uint16_t* lds) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < NB; b++) op_a[b].stage(lds + 16 * (2 + b) * D, (s * NW + wave) * D);
  };
  f32x4 acc[1 + NB];
#pragma unroll
  for (int b = 0; b <= NB; b++) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const uint16_t* lds) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < D / 32; kk++) {
      const bf16x8 fx = NarrowRows<16, D>::frag(lds, 0, kk, lane);
#pragma unroll
      for (int b = 0; b <= NB; b++)
        acc[b] = ET::mfma(NarrowRows<16, D>::frag(lds + 16 * (1 + b) * D, 0, kk, lane), fx, acc[b]);
    }
    wait_lds();   // read, before the next copies into this part
    asm volatile("" ::: "memory");
  };
  const int steps = (a.K + D * NW - 1) / (D * NW);
  issue_a(0, la);
  issue_a(1, lb);
  wait_vm<2 * NB>();   // in order of issue: x and W of both slices, A of the first
  asm volatile("" ::: "memory");
  for (int s = 0; s < steps; s += 2) {
    if (s) {
      wait_vm<kCopies>();
      asm volatile("" ::: "memory");
    }
    compute(la);
    issue_xw(s + 2, la);
    issue_a(s + 2, la);
    wait_vm<kCopies>();
    asm volatile("" ::: "memory");
    compute(lb);
    issue_xw(s + 3, lb);
    issue_a(s + 3, lb);
  }
  wait_vm<0>();   // no copy is left behind
  bf16x8 bv[NB];
  float scale[NB];
  if (wave == 0) {   // (the loads run while the sums are joined)
#pragma unroll
    for (int b = 0; b < NB; b++) {
      bv[b] = load_b(a, bad[b], brank[b], n, bfirst[b] + 8 * ((lane >> 4) & 1));
      scale[b] = brank[b] && a.scales ? a.scales[bad[b]] : 1.f;
    }
  }
  __syncthreads();
  f32x4(*s_part)[1 + NB][64] = reinterpret_cast<f32x4(*)[1 + NB][64]>(&s_a[0][0]);
#pragma unroll
  for (int b = 0; b <= NB; b++) s_part[wave][b][lane] = acc[b];
  __syncthreads();
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  static_assert(NB + 1 <= NW, "a wave per block of sums");
  if (wave <= NB) {
    v = s_part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < NW; w++) {
      const f32x4 q = s_part[w][wave][lane];
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] += q[e];
    }
  }
#pragma unroll
  for (int b = 0; b < NB; b++) {
    if (wave != b + 1 || !brank[b]) continue;
    // lane: token l % 16, ranks bfirst + 4 (l / 16) + 0..3
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < 4; q++) {
      if (bfirst[b] + 4 * (lane >> 4) + q >= brank[b]) v[q] = 0.f;
      m = fmaxf(m, fabsf(v[q]));
    }
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    const SplitV<ET> sv(m);
    // (fragment order: term, ranks 0..7 or 8..15, token, rank)
    uint16_t* out = &s_terms[b][128 * (lane >> 5) + 8 * t + 4 * ((lane >> 4) & 1)];
#pragma unroll
    for (int q = 0; q < 4; q++) sv.split(v[q], out + q);
    if (lane < 16) s_mul[b][t] = sv.up;
  }
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int b = 0; b < NB; b++) {
    if (!brank[b]) continue;
    const f32x4 d = times_v<ET>(bv[b], *reinterpret_cast<const bf16x8*>(&s_terms[b][8 * lane]),
                                *reinterpret_cast<const bf16x8*>(&s_terms[b][512 + 8 * lane]));
    if (id == bad[b]) {
      const float mul = s_mul[b][t] * scale[b];
#pragma unroll
      for (int q = 0; q < 4; q++) v[q] += mul * d[q];
    }
  }
  lora_store<ET>(a, t, n0 + 4 * (lane >> 4), v);
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
// index blocks of 16 tokens and 16 ranks
static inline size_t lora_blocks(int T, int rank_max) { return (size_t)((T + 15) / 16) * ((rank_max + 15) / 16); }

template <class ET, int NW, int D>
static hipError_t launch_skinny(const LoraArgs& a, hipStream_t s) {
  ProfScope prof("lora_linear", s);
  EXMOE_LAUNCH(prof, (lora_skinny_kernel<ET, NW, D>), dim3((a.N + 15) / 16, (a.T + 15) / 16), dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}
template <class ET, int TP, int TQ>
static hipError_t launch_mid(const LoraArgs& a, hipStream_t s) {
  const int tt = (a.T + 16 * TP - 1) / (16 * TP);
  ProfScope prof("lora_linear", s);
  EXMOE_LAUNCH(prof, (lora_mid_kernel<ET, TP, TQ>), dim3((a.N + 16 * TQ - 1) / (16 * TQ) * tt), dim3(256), 0, s, a, tt);
  return hipGetLastError();
}
template <class ET, int NB, int NW>
static hipError_t launch_token(const LoraArgs& a, hipStream_t s) {
  ProfScope prof("lora_linear", s);
  EXMOE_LAUNCH(prof, (lora_token_kernel<ET, NB, NW>), dim3((a.N + 15) / 16), dim3(64 * NW), 0, s, a);
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

template <class ET>
static hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int distinct = std::min(a.adapters, std::min(a.T, 16));   // adapters among 16 tokens, at most
  // one launch where every workgroup can make v itself (1 token, rank 16, 2048 x 2048: 7.5 us
  // against 9.9 us for two launches)
  if (a.T <= 16 && distinct * a.rank_blocks <= 4) {
    if (distinct * a.rank_blocks == 1) return launch_token<ET, 1, 8>(a, s);
    return launch_token<ET, 4, 5>(a, s);
  }
  {
    ProfScope prof("lora_shrink", s);
    EXMOE_LAUNCH(prof, (lora_shrink_kernel<ET, 4, 64>), dim3((a.T + 15) / 16, a.T > 256 ? std::min(distinct, 8) : distinct, a.rank_blocks),
                 dim3(256), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool span = 2 * ((size_t)(a.T - 1) * a.ldx + a.K) < kMaxSpan && 2 * ((size_t)(a.N - 1) * a.ldw + a.K) < kMaxSpan;
  // Pipelined 128 x 128 tiles against 64 x 64 blocks, one of which a compute unit holds: beyond
  // two rounds of those. K = 2048, ranks to 64, us: 1024 tokens of 512 requests, N = 2048 (512
  // blocks) 86 / 65, of 8 requests 40 / 35; 300 tokens of 20 requests, N = 5632 (440) 40 / 36; 600
  // tokens of 20 requests, N = 5632 (880) 41 / 56; 555 tokens, N = 3712, K = 7472 (522) 107 / 120.
  const long long blocks = (long long)((a.T + 63) / 64) * ((a.N + 63) / 64);
  if (a.w && span && a.T > 64 && blocks > 512) {
    if ((long long)((a.T + 255) / 256) * ((a.N + 255) / 256) >= 256) return launch_lora_wide<ET, 4, 2, 2, 4, 2>(a, s);
    return launch_lora_wide<ET, 2, 2, 2, 2, 2>(a, s);
  }
  // 64 x 64 blocks, then 32 x 32, against 16 x 16, where at least 100 of them share the chip, us:
  // 128 tokens of 128 requests, N = 5632 (176 of 64 x 64) 29 / 47; 94 tokens, N = 5664 (178) 25 / 40;
  // 64 tokens, N = 6400 (100), of 64 requests 40 / 42, of 4 requests 22 / 31; 40 tokens of 4, N = 8192
  // (128) 28 / 45, of 40, N = 6400 (100) 38 / 33; 256 tokens of 8 requests, N = 2048 (128) 25 / 34; 128
  // of 128 requests, N = 2048 (64) 40 / 27. 32 x 32: 155 tokens, N = 848 (135) 31 / 39; 3896 tokens,
  // N = 64 (244) 21 / 29; 100 tokens of 8 requests, N = 2048 (256) 15 / 20, 128 of 128 28 / 27.
  if (a.T > 32 && blocks >= 100) return launch_mid<ET, 4, 4>(a, s);
  if (a.T > 64 && (long long)((a.T + 31) / 32) * ((a.N + 31) / 32) >= 100) return launch_mid<ET, 2, 2>(a, s);
  return launch_skinny<ET, 8, 64>(a, s);
}

static int lora_shape(int T, int N, int K, int adapters, int rank_max) {
  if (T < 0 || T > (1 << 22)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "T must be in [0, 2^22] (got %d)", T);
  if (N < 1 || N > (1 << 20)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "N must be in [1, 2^20] (got %d)", N);
  if (K < 8 || K % 8 || K > (1 << 20)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "K must be a positive multiple of 8 up to 2^20 (got %d)", K);
  if (adapters < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "adapters must be positive (got %d)", adapters);
  if (rank_max < 8 || rank_max % 8 || rank_max > kMaxRank)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "rank_max must be a multiple of 8 in [8, 128] (got %d)", rank_max);
  // 64 x 64 blocks, which every large call can run on (16 x 16 and 32 x 32 blocks are for few)
  if ((long long)((T + 63) / 64) * ((N + 63) / 64) * 256 > 0xFFFFFF00ll)
    return set_error(EXMOE_ERR_UNSUPPORTED, "T x N has too many output tiles for one launch");
  return EXMOE_OK;
}

static int check_rows16(const char* name, const void* p, size_t ld, size_t stride, int cols) {
  if (!p) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if (!aligned16(p) || ld % 8 || stride % 8)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: rows must be 16-byte aligned", name);
  if (ld < (size_t)cols) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: row stride %zu smaller than its %d columns", name, ld, cols);
  if (ld > (1u << 24)) return set_error(EXMOE_ERR_UNSUPPORTED, "%s: row stride %zu larger than 2^24", name, ld);   // 16 rows: 32-bit offsets
  return EXMOE_OK;
}

}  // namespace exmoe

using namespace exmoe;

extern "C" size_t exmoe_lora_workspace_bytes(int T, int N, int K, int adapters, int rank_max) {
  if (lora_shape(T, N, K, adapters, rank_max)) return 0;
  return lora_blocks(T, rank_max) * (2048 + 64) + (size_t)T * 8;
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
  const bool many = bank->adapters > 1;   // (the stride of a single adapter means nothing)
  if ((st = check_rows16("bank->a", bank->a, bank->lda, many ? bank->a_stride : 0, K))) return st;
  if ((st = check_rows16("bank->b", bank->b, bank->ldb, many ? bank->b_stride : 0, bank->rank_max))) return st;
  if (many && (bank->a_stride < (size_t)(bank->rank_max - 1) * bank->lda + K ||
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
  const size_t L = (size_t)bank->adapters, R = (size_t)bank->rank_max;
  const MemRows mx = mem_matrix("x", x, T, ldx, K, 2), mw = mem_matrix("w", w, N, ldw, K, 2),
                ma = mem_matrices("bank->a", bank->a, L, bank->a_stride, R, bank->lda, K, 2),
                mb = mem_matrices("bank->b", bank->b, L, bank->b_stride, N, bank->ldb, R, 2),
                mr = mem_flat("bank->ranks", bank->ranks, L * 4), ms = mem_flat("bank->scales", bank->scales, L * 4),
                mi = mem_flat("adapter_ids", adapter_ids, (size_t)T * 4), my = mem_matrix("y", y, T, ldy, N, 2);
  if ((st = check_apart(my, {mx, mw, ma, mb, mr, ms, mi}))) return st;
  if ((st = check_apart(mem_flat("workspace", workspace, need), {mx, mw, ma, mb, mr, ms, mi, my}))) return st;
  LoraArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.w = static_cast<const uint16_t*>(w); a.ldx = ldx; a.ldw = ldw; a.ldy = ldy;
  a.a = static_cast<const uint16_t*>(bank->a); a.b = static_cast<const uint16_t*>(bank->b); a.lda = bank->lda;
  a.a_stride = bank->a_stride; a.ldb = bank->ldb; a.b_stride = bank->b_stride; a.ranks = bank->ranks;
  a.scales = bank->scales; a.ids = adapter_ids; a.adapters = bank->adapters; a.rank_max = bank->rank_max; a.T = T;
  a.N = N; a.K = K; a.y = static_cast<uint16_t*>(y); a.vec8 = (uintptr_t)y % 8 == 0 && ldy % 4 == 0;
  a.vec16 = aligned16(y) && ldy % 8 == 0; a.rank_blocks = (bank->rank_max + 15) / 16;
  a.terms = static_cast<uint16_t*>(workspace);
  a.mul = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + lora_blocks(T, bank->rank_max) * 2048);
  a.info = reinterpret_cast<int2*>(a.mul + lora_blocks(T, bank->rank_max) * 16);
  const hipError_t e = dtype == EXMOE_DTYPE_FP16 ? launch_lora<ElemFP16>(a, stream) : launch_lora<ElemBF16>(a, stream);
  return e == hipSuccess ? EXMOE_OK : hip_error(e, "exmoe_lora_linear");
}
