// Products grouped by expert over ragged segments of rows, and their gradients, gfx950.
//
//   forward        y[s, n]  = sum_k x[src(s), k] W_e[n, k]        s in segment e
//   gradient of x  dx[s, k] = sum_n dy[s, n] W_e[n, k]            (summed per token on request)
//   gradient of W  dW_e[n, k] = sum_{s in segment e} dy[s, n] x[src(s), k]
//
// Segments are offsets[e]..offsets[e + 1] of the rows sorted by expert (read on the device;
// clamped to [0, rows], so that no offset leads out of a buffer). One launch covers every
// expert: a workgroup finds its expert and tile from a scan of the offsets (E <= 256).
#include "grouped.h"

#include "exmoe.h"
#include "gemm_tile.h"

namespace exmoe {

enum { kMM = 0, kDG = 1, kWG = 2 };

struct RowTile {
  int e, seg0, cnt, p0, qt;
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Tile of workgroup b among ceil(count_e / BP) x q_tiles tiles per expert: all row tiles of
// one column tile follow each other (they read the same slice of W). Whole workgroup.
template <int BP>
__device__ bool resolve_rows(const int32_t* __restrict__ offsets, int rows, int E, int q_tiles, int b, RowTile& t,
                             int* s_scan, int* s_off) {
  const int tid = threadIdx.x;
  if (tid < 64) {
    int o[5];
#pragma unroll
    for (int q = 0; q < 5; q++) {
      const int e = tid * 4 + q;
      o[q] = offsets[e <= E ? e : E];
    }
    int v[4], run = 0;
#pragma unroll
    for (int q = 0; q < 5; q++) o[q] = clampi(o[q], 0, rows);
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int c = tid * 4 + q < E ? o[q + 1] - o[q] : 0;
      v[q] = c > 0 ? (c + BP - 1) / BP : 0;
      run += v[q];
      s_off[tid * 4 + q] = o[q];
    }
    if (tid == 63) s_off[kMaxExperts] = o[4];
    int incl = run;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(incl, off, 64);
      if (tid >= off) incl += u;
    }
    int ex = incl - run;
#pragma unroll
    for (int q = 0; q < 4; q++) {
      s_scan[tid * 4 + q] = ex;
      ex += v[q];
    }
    if (tid == 63) s_scan[kMaxExperts] = incl;
  }
  __syncthreads();
  const int total = s_scan[kMaxExperts] * q_tiles;
  if (b >= total) return false;
  const int idx = xcd_contiguous(b, total);
  int lo = 0, hi = E - 1;   // the largest e with scan[e] * q_tiles <= idx owns it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_scan[mid] * q_tiles <= idx) lo = mid; else hi = mid - 1;
  }
  t.e = lo;
  t.seg0 = s_off[lo];
  t.cnt = s_off[lo + 1] - t.seg0;
  const int np = (t.cnt + BP - 1) / BP;
  const int local = idx - s_scan[lo] * q_tiles;
  t.qt = local / np;
  t.p0 = (local - t.qt * np) * BP;
  return true;
}

// value / d for 0 <= value, d >= 1, with mul = floor((2^32 - 1) / d): the high product is
// the quotient or one less, and one compare corrects it.
__device__ __forceinline__ int div_by(int v, int d, uint32_t mul) {
  uint32_t q = __umulhi((uint32_t)v, mul);
  if ((uint32_t)v - q * (uint32_t)d >= (uint32_t)d) q++;
  return (int)q;
}

// One BP x BQ output tile per workgroup of WP x WQ waves, each owning a BP/WP x BQ/WQ part;
// 64-deep slices of both operands double-buffered in LDS, one barrier per slice.
template <class ET, int MODE, int BP, int BQ, int WP, int WQ, bool ALIGNED>
__global__ __launch_bounds__(64 * WP * WQ) void grouped_kernel(GroupedArgs a, int p_tiles, int q_tiles, int splits) {
  constexpr int NW = WP * WQ, TP = BP / WP / 16, TQ = BQ / WQ / 16;
  using OpP = std::conditional_t<MODE == kWG, ColOperand<BP, NW, ALIGNED>, RowOperand<BP, NW, ALIGNED>>;
  using OpQ = std::conditional_t<MODE == kMM, RowOperand<BQ, NW, ALIGNED>, ColOperand<BQ, NW, ALIGNED>>;
  __shared__ __attribute__((aligned(16))) uint16_t s_p0[BP * kBK], s_p1[BP * kBK], s_q0[BQ * kBK], s_q1[BQ * kBK];
  __shared__ int s_scan[kMaxExperts + 1], s_off[kMaxExperts + 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave / WQ, wq = wave % WQ;
  const int Q = MODE == kMM ? a.N : a.K;    // output columns
  const uint32_t dmul = 0xFFFFFFFFu / (uint32_t)a.row_div;

  int e, seg0, cnt, p0, q0, red, r_begin = 0, split = 0;
  if constexpr (MODE == kWG) {
    int idx = xcd_contiguous(blockIdx.x, gridDim.x);
    const int per = p_tiles * q_tiles;
    const int es = idx / per;
    idx -= es * per;
    e = es / splits;
    split = es - e * splits;
    p0 = idx / q_tiles * BP;
    q0 = idx % q_tiles * BQ;
    const int o0 = clampi(a.offsets[e], 0, a.rows), o1 = clampi(a.offsets[e + 1], 0, a.rows);
    seg0 = o0;
    cnt = o1 > o0 ? o1 - o0 : 0;
    const int steps = (cnt + kBK - 1) / kBK;
    r_begin = (int)((long long)steps * split / splits) * kBK;
    const int r_end = (int)((long long)steps * (split + 1) / splits) * kBK;
    seg0 += r_begin;
    cnt = (r_end < cnt ? r_end : cnt) - r_begin;
    if (cnt < 0) cnt = 0;
    red = cnt;
  } else {
    RowTile t;
    if (!resolve_rows<BP>(a.offsets, a.rows, a.E, q_tiles, blockIdx.x, t, s_scan, s_off)) return;
    e = t.e;
    seg0 = t.seg0;
    cnt = t.cnt;
    p0 = t.p0;
    q0 = t.qt * BQ;
    red = MODE == kMM ? a.K : a.N;
  }

  OpP op_p;
  OpQ op_q;
  if constexpr (MODE == kWG) {
    op_p.init(a.a + (size_t)seg0 * a.lda + p0, a.lda, red, a.N - p0);
    op_q.init(a.b + q0, a.ldb, red, a.K - q0);
  } else {
    // rows past the segment repeat its last one; an index outside x reads row 0 (such rows
    // are stored as zeros)
    op_p.init(a.a, red, wave, lane, [&](int i) {
      int s = seg0 + (p0 + i < cnt ? p0 + i : cnt - 1);
      if (MODE == kMM && a.row_index) {
        const int v = a.row_index[s];
        s = v < 0 ? a.x_rows : div_by(v, a.row_div, dmul);
        if (s >= a.x_rows) s = 0;
      } else if (MODE == kMM && s >= a.x_rows) {
        s = 0;
      }
      return (size_t)s * a.lda;
    });
    if constexpr (MODE == kMM) {
      op_q.init(a.b + (size_t)e * a.b_stride, red, wave, lane, [&](int i) {
        return (size_t)(q0 + i < Q ? q0 + i : Q - 1) * a.ldb;
      });
    } else {
      op_q.init(a.b + (size_t)e * a.b_stride + q0, a.ldb, red, Q - q0);
    }
  }

  // gradient of W: the rows of x behind the next slice's sorted rows, loaded a slice ahead
  int gidx[MODE == kWG ? OpQ::kSlots : 1];
  auto load_idx = [&](int k0) {
    if constexpr (MODE == kWG) {
#pragma unroll
      for (int i = 0; i < OpQ::kSlots; i++) {
        const int r = k0 + (i * NW + wave) * OpQ::kRows + lane / OpQ::kChunks;
        int v = seg0 + r;
        if (r < red && a.row_index) v = a.row_index[v];
        gidx[i] = v;
      }
    }
  };
  auto stage = [&](int k0, uint16_t* lp, uint16_t* lq) {
    if constexpr (MODE == kWG) {
      op_p.stage(lp, k0, wave, lane, [&](int r, int) { return (size_t)r * a.lda; });
      op_q.stage(lq, k0, wave, lane, [&](int, int i) {
        const int v = gidx[i];
        const int s = v < 0 ? a.x_rows : (a.row_index ? div_by(v, a.row_div, dmul) : v);
        return s < a.x_rows ? (size_t)s * a.ldb : ~(size_t)0;
      });
      load_idx(k0 + kBK);
    } else {
      op_p.stage(lp, k0, wave, lane);
      if constexpr (MODE == kMM) op_q.stage(lq, k0, wave, lane);
      else op_q.stage(lq, k0, wave, lane, [&](int r, int) { return (size_t)r * a.ldb; });
    }
  };

  f32x4 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = (red + kBK - 1) / kBK;
  auto step = [&](int s, const uint16_t* cp, const uint16_t* cq, uint16_t* np, uint16_t* nq) {
    __builtin_amdgcn_s_waitcnt(0);   // this slice has landed; everyone is past the last one
    __syncthreads();
    if (s + 1 < steps) stage((s + 1) * kBK, np, nq);
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
  if (steps > 0) {
    load_idx(0);
    stage(0, s_p0, s_q0);
    for (int s = 0; s < steps; s += 2) {
      step(s, s_p0, s_q0, s_p1, s_q1);
      if (s + 1 < steps) step(s + 1, s_p1, s_q1, s_p0, s_q0);
    }
  }

  // lane l holds p = l % 16 and q = 4 (l / 16) + 0..3 of each 16 x 16 part
  void* out = a.out;
  bool f32 = a.out_f32;
  size_t obase = 0, ldo = a.ldo;
  if (MODE == kWG) {
    if (splits > 1) {   // partial sums, [split][E][N][K]
      out = a.ws;
      f32 = true;
      ldo = (size_t)a.K;
      obase = ((size_t)split * a.E + e) * a.N * a.K;
    } else {
      obase = (size_t)e * a.o_stride;
    }
  }
  const bool vec = MODE == kWG && splits > 1 ? a.K % 4 == 0 : a.vec;
  const int plim = MODE == kWG ? a.N : cnt;
#pragma unroll
  for (int i = 0; i < TP; i++) {
    const int p = p0 + (wp * TP + i) * 16 + (lane & 15);
    if (p >= plim) continue;
    const size_t prow = MODE == kWG ? (size_t)p : (size_t)(seg0 + p);
    bool zero = false;
    if (MODE == kMM) {
      const int v = a.row_index ? a.row_index[prow] : (int)prow;
      zero = v < 0 || (a.row_index ? div_by(v, a.row_div, dmul) : v) >= a.x_rows;
    }
#pragma unroll
    for (int j = 0; j < TQ; j++) {
      const int q = q0 + (wq * TQ + j) * 16 + 4 * (lane >> 4);
      if (q < Q) store4<ET>(out, obase + prow * ldo + q, f32, vec, Q - q, zero ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[j][i]);
    }
  }
}

// dx[t, :] = sum_j rows[flat_to_sorted[t k + j], :] in slot order, rounded once. Entries
// outside the grouped rows add nothing. VEC columns per thread.
template <class ET, int VEC>
__global__ __launch_bounds__(256) void token_sum_kernel(const float* __restrict__ rows_ws, const int32_t* __restrict__ f2s,
                                                        const int32_t* __restrict__ offsets, int rows, int E, int T,
                                                        int K, int k, void* out, size_t ldo, int out_f32, int vec) {
  const int per = K / VEC;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (size_t)T * per) return;
  const int t = (int)(i / per), c = (int)(i - (size_t)t * per) * VEC;
  const int lo = clampi(offsets[0], 0, rows), hi = clampi(offsets[E], 0, rows);
  float v[VEC];
#pragma unroll
  for (int q = 0; q < VEC; q++) v[q] = 0.f;
  for (int j = 0; j < k; j++) {
    const int s = f2s[(size_t)t * k + j];
    if (s < lo || s >= hi) continue;
    const float* src = rows_ws + (size_t)s * K + c;
    if constexpr (VEC == 4) {
      const f32x4 r = *reinterpret_cast<const f32x4*>(src);
#pragma unroll
      for (int q = 0; q < 4; q++) v[q] += r[q];
    } else {
      v[0] += src[0];
    }
  }
  const size_t o = (size_t)t * ldo + c;
  if constexpr (VEC == 4)
    store4<ET>(out, o, out_f32, vec, 4, f32x4{v[0], v[1], v[2], v[3]});
  else if (out_f32)
    static_cast<float*>(out)[o] = v[0];
  else
    static_cast<uint16_t*>(out)[o] = ET::from_f32(v[0]);
}

// dW = sum of the partial sums in split order.
template <class ET>
__global__ __launch_bounds__(256) void split_sum_kernel(const float* __restrict__ part, int splits, int E, int N, int K,
                                                        void* out, size_t ldo, size_t o_stride, int out_f32) {
  const size_t n = (size_t)E * N * K;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
  for (int s = 0; s < splits; s++) v += part[(size_t)s * n + i];
  const size_t row = i / K, col = i - row * K, e = row / N;
  const size_t o = e * o_stride + (row - e * N) * ldo + col;
  if (out_f32) static_cast<float*>(out)[o] = v;
  else static_cast<uint16_t*>(out)[o] = ET::from_f32(v);
}

// ------------------------------------------------------------------------------------ host
static inline int ceil_div(int a, int b) { return (int)(((long long)a + b - 1) / b); }
constexpr long long kMaxThreads = 0xFFFFFFFFll;   // of one launch; larger calls are refused

// Parts into which the sum over an expert's rows is split: enough workgroups for the chip
// where an expert's gradient has few tiles, at least four 64-row slices per part.
static int wgrad_splits(int rows, int N, int K, int E) {
  const long long tiles = (long long)E * ceil_div(N, 128) * ceil_div(K, 128);
  const int avg = rows / E;
  long long s = 512 / (tiles > 0 ? tiles : 1);
  if (s > avg / 256) s = avg / 256;
  if (s > 16) s = 16;
  return s < 1 ? 1 : (int)s;
}

size_t grouped_workspace_bytes(int op, int rows, int N, int K, int E, int k) {
  if (op == EXMOE_GROUPED_DGRAD && k > 0) return (size_t)rows * K * 4;
  if (op == EXMOE_GROUPED_WGRAD) {
    const int s = wgrad_splits(rows, N, K, E);
    return s > 1 ? (size_t)s * E * N * K * 4 : 0;
  }
  return 0;
}

template <class ET, int MODE, int BP, int BQ, int WP, int WQ, bool ALIGNED>
static hipError_t launch_rows(const GroupedArgs& a, const char* name, hipStream_t s) {
  const long long max_p = a.rows / BP + (a.E < a.rows ? a.E : a.rows);
  const int qt = ceil_div(MODE == kMM ? a.N : a.K, BQ);
  if (max_p * qt * (64 * WP * WQ) > kMaxThreads) return hipErrorInvalidConfiguration;
  ProfScope prof(name, s);
  EXMOE_LAUNCH(prof, (grouped_kernel<ET, MODE, BP, BQ, WP, WQ, ALIGNED>), dim3((unsigned)(max_p * qt)),
               dim3(64 * WP * WQ), 0, s, a, 0, qt, 1);
  return hipGetLastError();
}

static bool op_aligned(const void* p, size_t ld, size_t stride, int len) {
  return aligned16(p) && ld % 8 == 0 && stride % 8 == 0 && len % 8 == 0;
}

template <class ET>
static hipError_t mm_type(const GroupedArgs& a, hipStream_t s) {
  const bool al = op_aligned(a.a, a.lda, 0, a.K) && op_aligned(a.b, a.ldb, a.b_stride, a.K);
  if (al) return launch_rows<ET, kMM, 128, 128, 2, 2, true>(a, "grouped_mm", s);
  return launch_rows<ET, kMM, 128, 128, 2, 2, false>(a, "grouped_mm", s);
}

hipError_t launch_grouped_mm(const GroupedArgs& a, hipStream_t s) {
  return a.fp16 ? mm_type<ElemFP16>(a, s) : mm_type<ElemBF16>(a, s);
}

template <class ET>
static hipError_t dgrad_type(const GroupedArgs& a, hipStream_t s) {
  const bool al = op_aligned(a.a, a.lda, 0, a.N) && op_aligned(a.b, a.ldb, a.b_stride, a.K);
  GroupedArgs r = a;
  if (a.flat_to_sorted) {
    if ((long long)(a.rows / a.k) * a.K > kMaxThreads) return hipErrorInvalidConfiguration;
    r.out = a.ws;
    r.vec = a.K % 4 == 0;
    r.ldo = (size_t)a.K;
    r.out_f32 = 1;
  }
  hipError_t e = al ? launch_rows<ET, kDG, 128, 128, 2, 2, true>(r, "grouped_dgrad", s)
                    : launch_rows<ET, kDG, 128, 128, 2, 2, false>(r, "grouped_dgrad", s);
  if (e != hipSuccess || !a.flat_to_sorted) return e;
  const int T = a.rows / a.k;
  ProfScope prof("token_sum", s);
  if (a.K % 4 == 0) {
    const size_t n = (size_t)T * (a.K / 4);
    EXMOE_LAUNCH(prof, (token_sum_kernel<ET, 4>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.ws,
                 a.flat_to_sorted, a.offsets, a.rows, a.E, T, a.K, a.k, a.out, a.ldo, a.out_f32, a.vec);
  } else {
    const size_t n = (size_t)T * a.K;
    EXMOE_LAUNCH(prof, (token_sum_kernel<ET, 1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.ws,
                 a.flat_to_sorted, a.offsets, a.rows, a.E, T, a.K, a.k, a.out, a.ldo, a.out_f32, a.vec);
  }
  return hipGetLastError();
}

hipError_t launch_grouped_dgrad(const GroupedArgs& a, hipStream_t s) {
  return a.fp16 ? dgrad_type<ElemFP16>(a, s) : dgrad_type<ElemBF16>(a, s);
}

template <class ET, bool ALIGNED>
static hipError_t wgrad_tiles(const GroupedArgs& a, hipStream_t s) {
  const int pt = ceil_div(a.N, 128), qt = ceil_div(a.K, 128), splits = wgrad_splits(a.rows, a.N, a.K, a.E);
  const long long grid = (long long)pt * qt * a.E * splits;
  if (grid * 256 > kMaxThreads) return hipErrorInvalidConfiguration;
  {
    ProfScope prof("grouped_wgrad", s);
    EXMOE_LAUNCH(prof, (grouped_kernel<ET, kWG, 128, 128, 2, 2, ALIGNED>), dim3((unsigned)grid), dim3(256), 0, s, a, pt,
                 qt, splits);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const size_t n = (size_t)a.E * a.N * a.K;
  ProfScope prof("split_sum", s);
  EXMOE_LAUNCH(prof, (split_sum_kernel<ET>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.ws, splits, a.E, a.N,
               a.K, a.out, a.ldo, a.o_stride, a.out_f32);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s) {
  const bool al = op_aligned(a.a, a.lda, 0, a.N) && op_aligned(a.b, a.ldb, 0, a.K);
  if (a.fp16) return al ? wgrad_tiles<ElemFP16, true>(a, s) : wgrad_tiles<ElemFP16, false>(a, s);
  return al ? wgrad_tiles<ElemBF16, true>(a, s) : wgrad_tiles<ElemBF16, false>(a, s);
}

}  // namespace exmoe

using namespace exmoe;

// ------------------------------------------------------------------------------------ C ABI
static int grouped_shape(int rows, int N, int K, int E, int dtype, int out_dtype) {
  if (rows < 0 || rows > (1 << 30)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^30] (got %d)", rows);
  if (N < 1 || K < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "N and K must be positive (got %d, %d)", N, K);
  if (N > (1 << 24) || K > (1 << 24)) return set_error(EXMOE_ERR_UNSUPPORTED, "N and K must be <= 2^24");
  if (E < 1 || E > kMaxExperts) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "E must be in [1, 256] (got %d)", E);
  if (dtype != EXMOE_DTYPE_BF16 && dtype != EXMOE_DTYPE_FP16)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "dtype must be bf16 or fp16 (got %d)", dtype);
  if (out_dtype != dtype && out_dtype != EXMOE_DTYPE_FP32)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "out_dtype must be dtype or fp32 (got %d)", out_dtype);
  return EXMOE_OK;
}

static int check_matrix(const char* name, const void* p, size_t ld, int cols, int bytes) {
  if (!p) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if ((uintptr_t)p % (unsigned)bytes) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must be %d-byte aligned", name, bytes);
  if (ld < (size_t)cols) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: row stride %zu smaller than its %d columns", name, ld, cols);
  return EXMOE_OK;
}

static int check_experts(const char* name, size_t ld, size_t stride, int N, int K, int E) {
  if (E > 1 && stride < (size_t)(N - 1) * ld + K)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: expert stride %zu smaller than a matrix", name, stride);
  return EXMOE_OK;
}

static int check_int32(const char* name, const void* p, bool may_be_null) {
  if (!p && !may_be_null) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if ((uintptr_t)p % 4) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must be 4-byte aligned", name);
  return EXMOE_OK;
}

static int check_ws(size_t need, const void* ws, size_t ws_bytes) {
  if (!need) return EXMOE_OK;
  if (!ws || ws_bytes < need)
    return set_error(EXMOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : 0);
  if (!aligned16(ws)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
  return EXMOE_OK;
}

static int launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return EXMOE_OK;
  if (e == hipErrorInvalidConfiguration) return set_error(EXMOE_ERR_UNSUPPORTED, "%s: too many output tiles for one launch", what);
  return hip_error(e, what);
}

// Whether four consecutive outputs of a row can be stored at once.
static int vec_store(const void* p, size_t ld, size_t stride, int out_f32) {
  return (uintptr_t)p % (out_f32 ? 16 : 8) == 0 && ld % 4 == 0 && stride % 4 == 0;
}

#define EXMOE_TRY(call)        \
  do {                         \
    const int st_ = (call);    \
    if (st_) return st_;       \
  } while (0)

extern "C" size_t exmoe_grouped_mm_workspace_bytes(int op, int rows, int N, int K, int E, int k) {
  if (op < EXMOE_GROUPED_MM || op > EXMOE_GROUPED_WGRAD || k < 0) {
    set_error(EXMOE_ERR_INVALID_ARGUMENT, "unknown grouped operator %d or negative k %d", op, k);
    return 0;
  }
  if (grouped_shape(rows, N, K, E, EXMOE_DTYPE_BF16, EXMOE_DTYPE_BF16)) return 0;
  return grouped_workspace_bytes(op, rows, N, K, E, k);
}

extern "C" int exmoe_grouped_mm(const void* x, size_t ldx, int x_rows, const int32_t* row_index, int row_div,
                                const int32_t* expert_offsets, const void* w, size_t ldw, size_t w_stride, int rows,
                                int N, int K, int E, int dtype, int out_dtype, void* y, size_t ldy, void* workspace,
                                size_t ws_bytes, hipStream_t stream) {
  EXMOE_TRY(grouped_shape(rows, N, K, E, dtype, out_dtype));
  if (row_div < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "row_div must be positive (got %d)", row_div);
  if (rows == 0) return EXMOE_OK;
  const int ob = out_dtype == EXMOE_DTYPE_FP32 ? 4 : 2;
  if (x_rows < (row_index ? 1 : rows))
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "x has %d rows, at least %d needed", x_rows, row_index ? 1 : rows);
  EXMOE_TRY(check_matrix("x", x, ldx, K, 2));
  EXMOE_TRY(check_matrix("w", w, ldw, K, 2));
  EXMOE_TRY(check_experts("w", ldw, w_stride, N, K, E));
  EXMOE_TRY(check_matrix("y", y, ldy, N, ob));
  EXMOE_TRY(check_int32("row_index", row_index, true));
  EXMOE_TRY(check_int32("expert_offsets", expert_offsets, false));
  EXMOE_TRY(check_ws(grouped_workspace_bytes(EXMOE_GROUPED_MM, rows, N, K, E, 0), workspace, ws_bytes));
  GroupedArgs a{};
  a.a = static_cast<const uint16_t*>(x); a.b = static_cast<const uint16_t*>(w); a.lda = ldx; a.ldb = ldw;
  a.b_stride = w_stride; a.offsets = expert_offsets; a.row_index = row_index; a.row_div = row_div; a.x_rows = x_rows;
  a.rows = rows; a.N = N; a.K = K; a.E = E; a.out = y; a.ldo = ldy; a.fp16 = dtype == EXMOE_DTYPE_FP16;
  a.out_f32 = ob == 4; a.vec = vec_store(y, ldy, 0, a.out_f32); a.ws = static_cast<float*>(workspace);
  return launched(launch_grouped_mm(a, stream), "exmoe_grouped_mm");
}

extern "C" int exmoe_grouped_mm_dgrad(const void* dy, size_t lddy, const int32_t* expert_offsets, const void* w,
                                      size_t ldw, size_t w_stride, const int32_t* flat_to_sorted, int k, int rows,
                                      int N, int K, int E, int dtype, int out_dtype, void* dx, size_t lddx,
                                      void* workspace, size_t ws_bytes, hipStream_t stream) {
  EXMOE_TRY(grouped_shape(rows, N, K, E, dtype, out_dtype));
  if (flat_to_sorted && (k < 1 || rows % k))
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "rows (%d) must be a multiple of k >= 1 (got %d)", rows, k);
  if (rows == 0) return EXMOE_OK;
  const int ob = out_dtype == EXMOE_DTYPE_FP32 ? 4 : 2;
  EXMOE_TRY(check_matrix("dy", dy, lddy, N, 2));
  EXMOE_TRY(check_matrix("w", w, ldw, K, 2));
  EXMOE_TRY(check_experts("w", ldw, w_stride, N, K, E));
  EXMOE_TRY(check_matrix("dx", dx, lddx, K, ob));
  EXMOE_TRY(check_int32("expert_offsets", expert_offsets, false));
  EXMOE_TRY(check_int32("flat_to_sorted", flat_to_sorted, true));
  EXMOE_TRY(check_ws(grouped_workspace_bytes(EXMOE_GROUPED_DGRAD, rows, N, K, E, flat_to_sorted ? k : 0), workspace,
                     ws_bytes));
  GroupedArgs a{};
  a.a = static_cast<const uint16_t*>(dy); a.b = static_cast<const uint16_t*>(w); a.lda = lddy; a.ldb = ldw;
  a.b_stride = w_stride; a.offsets = expert_offsets; a.row_div = 1; a.x_rows = rows; a.rows = rows; a.N = N; a.K = K;
  a.E = E; a.out = dx; a.ldo = lddx; a.fp16 = dtype == EXMOE_DTYPE_FP16; a.out_f32 = ob == 4;
  a.vec = vec_store(dx, lddx, 0, a.out_f32); a.flat_to_sorted = flat_to_sorted; a.k = k;
  a.ws = static_cast<float*>(workspace);
  return launched(launch_grouped_dgrad(a, stream), "exmoe_grouped_mm_dgrad");
}

extern "C" int exmoe_grouped_mm_wgrad(const void* dy, size_t lddy, const void* x, size_t ldx, int x_rows,
                                      const int32_t* row_index, int row_div, const int32_t* expert_offsets, int rows,
                                      int N, int K, int E, int dtype, int out_dtype, void* dw, size_t lddw,
                                      size_t dw_stride, void* workspace, size_t ws_bytes, hipStream_t stream) {
  EXMOE_TRY(grouped_shape(rows, N, K, E, dtype, out_dtype));
  if (row_div < 1) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "row_div must be positive (got %d)", row_div);
  const int ob = out_dtype == EXMOE_DTYPE_FP32 ? 4 : 2;
  if (rows > 0) {
    if (x_rows < (row_index ? 1 : rows))
      return set_error(EXMOE_ERR_INVALID_ARGUMENT, "x has %d rows, at least %d needed", x_rows, row_index ? 1 : rows);
    EXMOE_TRY(check_matrix("dy", dy, lddy, N, 2));
    EXMOE_TRY(check_matrix("x", x, ldx, K, 2));
  }
  EXMOE_TRY(check_matrix("dw", dw, lddw, K, ob));
  EXMOE_TRY(check_experts("dw", lddw, dw_stride, N, K, E));
  EXMOE_TRY(check_int32("row_index", row_index, true));
  EXMOE_TRY(check_int32("expert_offsets", expert_offsets, false));
  EXMOE_TRY(check_ws(grouped_workspace_bytes(EXMOE_GROUPED_WGRAD, rows, N, K, E, 0), workspace, ws_bytes));
  GroupedArgs a{};
  a.a = static_cast<const uint16_t*>(dy); a.b = static_cast<const uint16_t*>(x); a.lda = lddy; a.ldb = ldx;
  a.offsets = expert_offsets; a.row_index = row_index; a.row_div = row_div; a.x_rows = x_rows; a.rows = rows; a.N = N;
  a.K = K; a.E = E; a.out = dw; a.ldo = lddw; a.o_stride = dw_stride; a.fp16 = dtype == EXMOE_DTYPE_FP16;
  a.out_f32 = ob == 4; a.vec = vec_store(dw, lddw, dw_stride, a.out_f32); a.ws = static_cast<float*>(workspace);
  return launched(launch_grouped_wgrad(a, stream), "exmoe_grouped_mm_wgrad");
}
