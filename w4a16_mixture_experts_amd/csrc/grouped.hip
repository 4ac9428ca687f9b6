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

#include "checks.h"
#include "exmoe.h"
#include "gemm_wide.h"
#include "overlap.h"
#include "row_tiles.h"

namespace exmoe {

enum { kMM = 0, kDG = 1, kWG = 2 };

// The tile of a workgroup: expert e, whose rows start at seg0 of the sorted order; rows
// p0..cnt of them (gradient of W: the cnt rows of this part of the sum, output rows from p0),
// columns from q0, length red of the summed axis.
struct TilePlace {
  int e, seg0, cnt, p0, q0, red, split;
};

template <int MODE, int BP, int BQ>
__device__ __forceinline__ bool place_tile(const GroupedArgs& a, int p_tiles, int q_tiles, int splits, TilePlace& t) {
  t.split = 0;
  if constexpr (MODE == kWG) {
    int idx = xcd_contiguous(blockIdx.x, gridDim.x);
    const int per = p_tiles * q_tiles;
    const int es = idx / per;
    idx -= es * per;
    t.e = es / splits;
    t.split = es - t.e * splits;
    int pt, qt;
    band_order(idx, p_tiles, q_tiles, pt, qt);
    t.p0 = pt * BP;
    t.q0 = qt * BQ;
    t.seg0 = clampi(a.offsets[t.e], 0, a.rows);
    const int o1 = clampi(a.offsets[t.e + 1], 0, a.rows);
    t.cnt = o1 > t.seg0 ? o1 - t.seg0 : 0;
    const int steps = (t.cnt + kBK - 1) / kBK;
    const int r_begin = (int)((long long)steps * t.split / splits) * kBK;
    const int r_end = (int)((long long)steps * (t.split + 1) / splits) * kBK;
    t.seg0 += r_begin;
    t.cnt = (r_end < t.cnt ? r_end : t.cnt) - r_begin;
    if (t.cnt < 0) t.cnt = 0;
    t.red = t.cnt;
  } else {
    RowTile r;
    if (!resolve_rows<BP>(a.offsets, a.rows, a.E, q_tiles, blockIdx.x, r)) return false;
    t.e = r.e;
    t.seg0 = r.seg0;
    t.cnt = r.p1;
    t.p0 = r.p0;
    t.q0 = r.qt * BQ;
    t.red = MODE == kMM ? a.K : a.N;
  }
  return true;
}

// Where a tile's outputs go: the caller's matrix, or the partial sums [split][E][N][K].
template <int MODE>
__device__ __forceinline__ TileOut tile_out(const GroupedArgs& a, const TilePlace& t, int splits) {
  TileOut o{a.out, 0, a.ldo, a.out_f32 != 0, a.vec != 0};
  if (MODE == kWG) {
    if (splits > 1) o = TileOut{a.ws, ((size_t)t.split * a.E + t.e) * a.N * a.K, (size_t)a.K, true, a.K % 4 == 0};
    else o.base = (size_t)t.e * a.o_stride;
  }
  return o;
}

// The simple form's operands and the staging of a slice.
template <int MODE, class OpP, class OpQ, int BP, int BQ, int NW>
struct TileWork {
  const GroupedArgs& a;
  int wave, lane, Q;
  uint32_t dmul;
  TilePlace t;
  OpP op_p;
  OpQ op_q;
  // gradient of W: the rows of x behind a slice's sorted rows, loaded a slice ahead
  int gidx[MODE == kWG ? OpQ::kSlots : 1];

  __device__ __forceinline__ TileWork(const GroupedArgs& args, int wave_, int lane_)
      : a(args), wave(wave_), lane(lane_), Q(MODE == kMM ? args.N : args.K), dmul(0xFFFFFFFFu / (uint32_t)args.row_div) {}

  __device__ __forceinline__ bool resolve(int p_tiles, int q_tiles, int splits) {
    if (!place_tile<MODE, BP, BQ>(a, p_tiles, q_tiles, splits, t)) return false;
    if constexpr (MODE == kWG) {
      op_p.init(a.a + (size_t)t.seg0 * a.lda + t.p0, a.lda, t.red, a.N - t.p0);
      op_q.init(a.b + t.q0, a.ldb, t.red, a.K - t.q0);
    } else {
      // rows past the segment repeat its last one; an index outside x reads row 0 (such rows
      // are stored as zeros)
      op_p.init(a.a, t.red, wave, lane, [&](int i) {
        int s = t.seg0 + (t.p0 + i < t.cnt ? t.p0 + i : t.cnt - 1);
        if (MODE == kMM) {
          if (a.row_index) {
            const int v = a.row_index[s];
            s = v < 0 ? a.x_rows : div_by(v, a.row_div, dmul);
          }
          if (s >= a.x_rows) s = 0;
        }
        return (size_t)s * a.lda;
      });
      if constexpr (MODE == kMM) {
        op_q.init(a.b + (size_t)t.e * a.b_stride, t.red, wave, lane,
                  [&](int i) { return (size_t)(t.q0 + i < Q ? t.q0 + i : Q - 1) * a.ldb; });
      } else {
        op_q.init(a.b + (size_t)t.e * a.b_stride + t.q0, a.ldb, t.red, Q - t.q0);
      }
    }
    return true;
  }

  __device__ __forceinline__ void load_idx(int k0) {
    if constexpr (MODE == kWG) {
#pragma unroll
      for (int i = 0; i < OpQ::kSlots; i++) {
        const int r = k0 + (i * NW + wave) * OpQ::kRows + lane / OpQ::kChunks;
        int v = t.seg0 + r;
        if (r < t.red && a.row_index) v = a.row_index[v];
        gidx[i] = v;
      }
    }
  }
  // element offset of a row of the Q operand when its summed axis is outermost (gradient of
  // W: of the rows of load_idx(k0))
  __device__ __forceinline__ size_t q_row(int r, int i) const {
    if constexpr (MODE == kWG) {
      const int v = gidx[i];
      const int s = v < 0 ? a.x_rows : (a.row_index ? div_by(v, a.row_div, dmul) : v);
      return s < a.x_rows ? (size_t)s * a.ldb : ~(size_t)0;
    }
    return (size_t)r * a.ldb;
  }
  // copies of a slice straight into LDS (aligned operands)
  __device__ __forceinline__ void stage(int k0, uint16_t* lp, uint16_t* lq) const {
    if constexpr (MODE == kWG) op_p.stage(lp, k0, wave, lane, [&](int r, int) { return (size_t)r * a.lda; });
    else op_p.stage(lp, k0, wave, lane);
    if constexpr (MODE == kMM) op_q.stage(lq, k0, wave, lane);
    else op_q.stage(lq, k0, wave, lane, [&](int r, int i) { return q_row(r, i); });
  }
  // or through registers: the loads, and later the values to LDS
  __device__ __forceinline__ void fetch(int k0, Any8 (&rp)[OpP::kSlots], Any8 (&rq)[OpQ::kSlots]) const {
    if constexpr (MODE == kWG) op_p.fetch(rp, k0, wave, lane, [&](int r, int) { return (size_t)r * a.lda; });
    else op_p.fetch(rp, k0, wave, lane);
    if constexpr (MODE == kMM) op_q.fetch(rq, k0, wave, lane);
    else op_q.fetch(rq, k0, wave, lane, [&](int r, int i) { return q_row(r, i); });
  }
  __device__ __forceinline__ void commit(const Any8 (&rp)[OpP::kSlots], const Any8 (&rq)[OpQ::kSlots], uint16_t* lp,
                                         uint16_t* lq) const {
    op_p.commit(rp, lp, wave, lane);
    op_q.commit(rq, lq, wave, lane);
  }
  // whether row p of x lies outside x (its outputs are zeros)
  __device__ __forceinline__ bool zero_row(int p) const {
    if (MODE != kMM) return false;
    const int v = a.row_index ? a.row_index[t.seg0 + p] : t.seg0 + p;
    return v < 0 || (a.row_index ? div_by(v, a.row_div, dmul) : v) >= a.x_rows;
  }
};

// One BP x BQ output tile per workgroup of WP x WQ waves, each owning a BP/WP x BQ/WQ part;
// 64-deep slices of both operands double-buffered in LDS, one barrier per slice. The form
// for operands of any alignment (through registers, fetched while the slice before runs) and
// for aligned ones that 32-bit offsets do not span (ALIGNED).
template <class ET, int MODE, int BP, int BQ, int WP, int WQ, bool ALIGNED>
__global__ __launch_bounds__(64 * WP * WQ) void grouped_kernel(GroupedArgs a, int p_tiles, int q_tiles, int splits) {
  constexpr int NW = WP * WQ, TP = BP / WP / 16, TQ = BQ / WQ / 16;
  using OpP = std::conditional_t<MODE == kWG, ColOperand<BP, NW>, RowOperand<BP, NW>>;
  using OpQ = std::conditional_t<MODE == kMM, RowOperand<BQ, NW>, ColOperand<BQ, NW>>;
  __shared__ __attribute__((aligned(16))) uint16_t s_p0[BP * kBK], s_p1[BP * kBK], s_q0[BQ * kBK], s_q1[BQ * kBK];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave / WQ, wq = wave % WQ;
  TileWork<MODE, OpP, OpQ, BP, BQ, NW> t(a, wave, lane);
  if (!t.resolve(p_tiles, q_tiles, splits)) return;

  f32x4 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = (t.t.red + kBK - 1) / kBK;
  Any8 rp[ALIGNED ? 1 : OpP::kSlots], rq[ALIGNED ? 1 : OpQ::kSlots];
  auto step = [&](int s, const uint16_t* cp, const uint16_t* cq, uint16_t* np, uint16_t* nq) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0);   // this slice has landed; everyone is past the last one
    __syncthreads();
    if (s + 1 < steps) {
      if constexpr (ALIGNED) t.stage((s + 1) * kBK, np, nq);
      else t.fetch((s + 1) * kBK, rp, rq);
      t.load_idx((s + 2) * kBK);
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
    if constexpr (!ALIGNED) {
      if (s + 1 < steps) t.commit(rp, rq, np, nq);
    }
  };
  if (steps > 0) {
    t.load_idx(0);
    if constexpr (ALIGNED) {
      t.stage(0, s_p0, s_q0);
    } else {
      t.fetch(0, rp, rq);
      t.commit(rp, rq, s_p0, s_q0);
    }
    t.load_idx(kBK);
    for (int s = 0; s < steps; s += 2) {
      step(s, s_p0, s_q0, s_p1, s_q1);
      if (s + 1 < steps) step(s + 1, s_p1, s_q1, s_p0, s_q0);
    }
  }

  // lane l holds p = l % 16 and q = 4 (l / 16) + 0..3 of each 16 x 16 part
  const TileOut out = tile_out<MODE>(a, t.t, splits);
  const int plim = MODE == kWG ? a.N : t.t.cnt;
#pragma unroll
  for (int i = 0; i < TP; i++) {
    const int p = t.t.p0 + (wp * TP + i) * 16 + (lane & 15);
    if (p >= plim) continue;
    const bool zero = t.zero_row(p);
    const size_t row = out.base + (size_t)(MODE == kWG ? p : t.t.seg0 + p) * out.ld;
#pragma unroll
    for (int j = 0; j < TQ; j++) {
      const int q = t.t.q0 + (wq * TQ + j) * 16 + 4 * (lane >> 4);
      if (q < t.Q)
        store4<ET>(out.ptr, row + q, out.f32, out.vec, t.Q - q, zero ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[j][i]);
    }
  }
}

// The pipelined form for aligned operands (gemm_wide.h).
template <class ET, int MODE, int TP, int TQ, int WP, int WQ, int D, int OCC>
__global__ __launch_bounds__(64 * WP * WQ, OCC) void grouped_wide_kernel(GroupedArgs a, int p_tiles, int q_tiles,
                                                                        int splits) {
  constexpr int NW = WP * WQ, BP = 32 * TP * WP, BQ = 32 * TQ * WQ;
  using OpP = std::conditional_t<MODE == kWG, WideCols<BP, NW, D>, WideRows<BP, NW, D>>;
  using OpQ = std::conditional_t<MODE == kMM, WideRows<BQ, NW, D>, WideCols<BQ, NW, D>>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  TilePlace t;
  if (!place_tile<MODE, BP, BQ>(a, p_tiles, q_tiles, splits, t)) return;
  const int Q = MODE == kMM ? a.N : a.K;
  const uint32_t dmul = 0xFFFFFFFFu / (uint32_t)a.row_div;
  OpP op_p;
  OpQ op_q;
  if constexpr (MODE == kWG) {
    op_p.template init<false>(make_buf(a.a + (size_t)t.seg0 * a.lda + t.p0, t.red ? 2 * ((t.red - 1) * a.lda + (a.len_a - t.p0)) : 0),
              2 * (uint32_t)a.lda, t.red, a.len_a - t.p0, wave, lane);
    op_q.template init<true>(make_buf(a.b + t.q0, a.x_rows ? 2 * ((a.x_rows - 1) * a.ldb + (a.len_b - t.q0)) : 0),
                                 2 * (uint32_t)a.ldb, t.red, a.len_b - t.q0, wave, lane);
  } else {
    const int rows_a = MODE == kMM ? a.x_rows : a.rows;
    op_p.init(make_buf(a.a, 2 * ((rows_a - 1) * a.lda + a.len_a)), t.red, wave, lane, [&](int i) {
      int s = t.seg0 + t.p0 + i;
      bool ok = t.p0 + i < t.cnt;
      if (MODE == kMM && a.row_index) {
        const int v = ok ? a.row_index[s] : -1;
        s = v < 0 ? a.x_rows : div_by(v, a.row_div, dmul);
        ok = s < a.x_rows;
      }
      return ok ? (uint32_t)((size_t)s * a.lda * 2) : kNowhere;
    });
    const uint16_t* w = a.b + (size_t)t.e * a.b_stride;
    if constexpr (MODE == kMM) {
      op_q.init(make_buf(w, 2 * ((a.N - 1) * a.ldb + a.len_b)), t.red, wave, lane, [&](int i) {
        return t.q0 + i < Q ? (uint32_t)((size_t)(t.q0 + i) * a.ldb * 2) : kNowhere;
      });
    } else {
      op_q.template init<false>(make_buf(w + t.q0, 2 * ((a.N - 1) * a.ldb + (a.len_b - t.q0))), 2 * (uint32_t)a.ldb, t.red, a.len_b - t.q0,
                wave, lane);
    }
  }
  wide_tile<ET, TP, TQ, WP, WQ, D, MODE == kWG>(
      op_p, op_q, t.red, t.p0, MODE == kWG ? a.N : t.cnt, t.q0, Q, tile_out<MODE>(a, t, splits),
      [&](int r) { return a.row_index ? a.row_index[t.seg0 + r] : t.seg0 + r; },
      [&](int v) {
        const int s = a.row_index ? div_by(v, a.row_div, dmul) : v;
        return s < a.x_rows ? (uint32_t)s * 2 * (uint32_t)a.ldb : kNowhere;
      },
      [](int, int, auto&) {}, [&](int p) { return MODE == kWG ? p : t.seg0 + p; });
}

// The forward product for few rows per expert, or few tiles: 16 TP rows x 16 TQ columns per
// workgroup, the waves split K (gemm_wide.h, narrow_product). TP = TQ = 1 is bound by reading
// W, which streams through once; 4 x 4 blocks shorten the loop of small products.
template <class ET, int TP, int TQ, int NW, int D, bool ALIGNED>
__global__ __launch_bounds__(64 * NW) void grouped_narrow_kernel(GroupedArgs a, int q_tiles) {
  constexpr int kPart = ALIGNED ? 16 * (TP + TQ) * D : TP * TQ * 64 * 4;   // (elements; the sums at least)
  __shared__ __attribute__((aligned(16))) uint16_t s_a[2][NW][kPart];        // two slices a wave
  static_assert(sizeof(f32x4) * TP * TQ * 64 * NW <= sizeof(s_a), "the sums fit into the slices' part");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile r;
  if (!resolve_rows<16 * TP, 16>(a.offsets, a.rows, a.E, q_tiles, blockIdx.x, r)) return;
  const int n0 = 16 * TQ * r.qt;
  const uint32_t dmul = 0xFFFFFFFFu / (uint32_t)a.row_div;
  // row i of the tile: its row of x, or -1
  auto source = [&](int i) {
    const int p = r.p0 + i;
    if (p >= r.p1) return -1;
    int s = r.seg0 + p;
    if (a.row_index) {
      const int v = a.row_index[s];
      s = v < 0 ? -1 : div_by(v, a.row_div, dmul);
    }
    return s < a.x_rows ? s : -1;
  };
  f32x4 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint16_t* w = a.b + (size_t)r.e * a.b_stride;
  if constexpr (ALIGNED) {
    using OpX = NarrowRows<16 * TP, D>;
    using OpW = NarrowRows<16 * TQ, D>;
    OpX op_x;
    OpW op_w;
    op_w.init(make_buf(w + (size_t)n0 * a.ldb, 2 * ((size_t)(min(16 * TQ, a.N - n0) - 1) * a.ldb + a.len_b)), a.K, lane,
              [&](int i) { return n0 + i < a.N ? (uint32_t)(i * a.ldb * 2) : kNowhere; });
    op_x.init(make_buf(a.a, 2 * ((size_t)(a.x_rows - 1) * a.lda + a.len_a)), a.K, lane, [&](int i) {
      const int s = source(i);
      return s < 0 ? kNowhere : (uint32_t)((size_t)s * a.lda * 2);
    });
    narrow_product<ET, TP, TQ, NW, D>(op_x, op_w, a.K, wave, lane, s_a[0][wave], s_a[1][wave], acc);
  } else {
    size_t xrow[TP], wrow[TQ];
    bool zero[TP];
#pragma unroll
    for (int j = 0; j < TQ; j++) wrow[j] = (size_t)min(n0 + 16 * j + (lane & 15), a.N - 1) * a.ldb;
#pragma unroll
    for (int i = 0; i < TP; i++) {
      const int s = source(16 * i + (lane & 15));
      zero[i] = s < 0;
      xrow[i] = zero[i] ? 0 : (size_t)s * a.lda;
    }
    skinny_product_any<ET, TP, TQ, NW>(a.a, xrow, w, wrow, a.K, wave, lane, acc);
#pragma unroll
    for (int i = 0; i < TP; i++)
#pragma unroll
      for (int j = 0; j < TQ; j++)
        if (zero[i]) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __syncthreads();
  f32x4 v[TQ];
  skinny_reduce<TP, TQ, NW>(reinterpret_cast<f32x4(*)[TQ * TP][64]>(&s_a[0][0][0]), acc, wave, lane, v);
  const int p = r.p0 + 16 * wave + (lane & 15);
  if (wave >= TP || p >= r.p1) return;
#pragma unroll
  for (int j = 0; j < TQ; j++) {
    const int q = n0 + 16 * j + 4 * (lane >> 4);
    if (q < a.N) store4<ET>(a.out, (size_t)(r.seg0 + p) * a.ldo + q, a.out_f32, a.vec, a.N - q, v[j]);
  }
}

// The gradient of x in the same way: 16 TP rows x 64 columns per workgroup, the waves split N.
template <class ET, int TP, int NW>
__global__ __launch_bounds__(64 * NW) void grouped_narrow_dgrad_kernel(GroupedArgs a, int q_tiles) {
  constexpr int D = 32, kPart = 16 * TP * D + 64 * D;
  using OpX = NarrowRows<16 * TP, D>;
  using OpW = NarrowCols<D>;
  __shared__ __attribute__((aligned(16))) uint16_t s_a[2][NW][kPart];   // two slices a wave
  static_assert(sizeof(f32x4) * TP * 4 * 64 * NW <= sizeof(s_a), "the sums fit into the slices' part");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile r;
  if (!resolve_rows<16 * TP, 16>(a.offsets, a.rows, a.E, q_tiles, blockIdx.x, r)) return;
  const int q0 = 64 * r.qt, p0 = r.seg0 + r.p0, cnt = r.p1 - r.p0;
  OpX op_x;
  OpW op_w;
  op_w.init(make_buf(a.b + (size_t)r.e * a.b_stride + q0, 2 * ((size_t)(a.N - 1) * a.ldb + (a.len_b - q0))),
            2 * (uint32_t)a.ldb, a.N, a.len_b - q0, lane);
  op_x.init(make_buf(a.a + (size_t)p0 * a.lda, 2 * ((size_t)(cnt - 1) * a.lda + a.len_a)), a.N, lane,
            [&](int i) { return i < cnt ? (uint32_t)(i * a.lda * 2) : kNowhere; });
  f32x4 acc[4][TP];
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int i = 0; i < TP; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  narrow_product<ET, TP, 4, NW, D>(op_x, op_w, a.N, wave, lane, s_a[0][wave], s_a[1][wave], acc);
  __syncthreads();
  f32x4 v[4];
  skinny_reduce<TP, 4, NW>(reinterpret_cast<f32x4(*)[4 * TP][64]>(&s_a[0][0][0]), acc, wave, lane, v);
  const int p = 16 * wave + (lane & 15);
  if (wave >= TP || p >= cnt) return;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int q = q0 + 16 * j + 4 * (lane >> 4);
    if (q < a.K) store4<ET>(a.out, (size_t)(p0 + p) * a.ldo + q, a.out_f32, a.vec, a.K - q, v[j]);
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

// Rows of len elements at any alignment into rows of pad (a multiple of 8) elements, zeros
// behind the len-th. Row r of group g comes from src + g stride + (row of r) ld, the row being
// r or row_index[r] / row_div (rows outside the src_rows of src: zeros). With offsets, group g
// is expert g, and experts without rows are left out. One thread per 8 elements.
__global__ __launch_bounds__(256) void pack_rows_kernel(const uint16_t* __restrict__ src, size_t ld, size_t stride, int len,
                                                        int rows, int src_rows, const int32_t* __restrict__ row_index,
                                                        int row_div, const int32_t* __restrict__ offsets,
                                                        uint16_t* __restrict__ dst, int pad) {
  const int per = pad / 8, g = blockIdx.y;
  if (offsets && offsets[g + 1] <= offsets[g]) return;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  const bool in = i < (size_t)rows * per;
  const int r = in ? (int)(i / per) : 0, c = in ? (int)(i - (size_t)r * per) * 8 : 0;
  int s = r;
  if (row_index) {
    const int v = row_index[r];
    s = v < 0 ? src_rows : div_by(v, row_div, 0xFFFFFFFFu / (uint32_t)row_div);
  }
  const bool ok = in && s < src_rows;
  const uint16_t* base = src + (size_t)g * stride;
  const size_t off = ok ? (size_t)s * ld + c : 0;
  Any8 v;
  if (__all(Any8::inner(base, off, len - c, ok))) v.fetch(base, off, ok);
  else v.fetch_edge(base, off, len - c, ok);
  if (in) *reinterpret_cast<uint4*>(dst + ((size_t)g * rows + r) * pad + c) = v.value();
}

// dW = sum of the partial sums in split order, VEC outputs of a row per thread.
template <class ET, int VEC>
__global__ __launch_bounds__(256) void split_sum_kernel(const float* __restrict__ part, int splits, int E, int N, int K,
                                                        void* out, size_t ldo, size_t o_stride, int out_f32, int vec) {
  const size_t n = (size_t)E * N * K;
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  if (i >= n) return;
  float v[VEC];
#pragma unroll
  for (int q = 0; q < VEC; q++) v[q] = 0.f;
#pragma unroll 8
  for (int s = 0; s < splits; s++) {
    if constexpr (VEC == 4) {
      const f32x4 r = *reinterpret_cast<const f32x4*>(part + (size_t)s * n + i);
#pragma unroll
      for (int q = 0; q < 4; q++) v[q] += r[q];
    } else {
      v[0] += part[(size_t)s * n + i];
    }
  }
  const size_t row = i / K, col = i - row * K, e = row / N;
  const size_t o = e * o_stride + (row - e * N) * ldo + col;
  if constexpr (VEC == 4)
    store4<ET>(out, o, out_f32, vec, 4, f32x4{v[0], v[1], v[2], v[3]});
  else if (out_f32)
    static_cast<float*>(out)[o] = v[0];
  else
    static_cast<uint16_t*>(out)[o] = ET::from_f32(v[0]);
}

// ------------------------------------------------------------------------------------ host
// Parts into which the sum over an expert's rows is split: enough workgroups for the chip
// where an expert's gradient has few tiles, at least four 64-row slices per part.
static int wgrad_splits(int rows, int N, int K, int E) {
  const long long tiles = (long long)E * ceil_div(N, 128) * ceil_div(K, 128);
  const int avg = rows / E;
  long long s = 384 / (tiles > 0 ? tiles : 1);
  if (s > avg / 256) s = avg / 256;
  if (s > 16) s = 16;
  return s < 1 ? 1 : (int)s;
}

static inline int pad8(int n) { return (n + 7) & ~7; }
static inline size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }
// Rows per expert from which the forward product copies operands with odd row lengths. Without
// and with copies, us: 22 experts of 3831 x 641, 16 rows 73 / 93, 30 rows 108 / 95, 41 rows 142 /
// 96, 84 rows 262 / 104; 13 experts of 517 x 1003, 31 rows 19 / 23, 39 rows 22 / 24, 60 rows 27 / 24.
// Skewed (Zipf), the 22 experts: 9 rows 56 / 91, 16 rows 73 / 92, 30 rows 107 / 97, 41 rows 138 / 96.
constexpr int kPackRows = 32;

// Operands whose rows are no multiple of 16 bytes long are copied with padded rows first, so
// that the products run on their aligned forms (one pass over the operand against loads
// through registers in the product: gradient of x, 1384 rows, N = 7827, K = 384: 510 -> 94 us).
// Not for the forward product's few rows per expert, which read W once or twice anyway.
GroupedWorkspace grouped_workspace(int op, int rows, int N, int K, int E, int k) {
  GroupedWorkspace w{0, 0, 0};
  const size_t rows_n = align16((size_t)rows * pad8(N) * 2), rows_k = align16((size_t)rows * pad8(K) * 2),
               weights = align16((size_t)E * N * pad8(K) * 2);
  if (op == EXMOE_GROUPED_MM) {
    if (K % 8 && rows > kPackRows * (long long)E) w.pack_a = rows_k, w.pack_b = weights;
  } else if (op == EXMOE_GROUPED_DGRAD) {
    if (k > 0) w.sums = align16((size_t)rows * K * 4);
    if (N % 8) w.pack_a = rows_n;
    if (K % 8) w.pack_b = weights;
  } else {
    const int s = wgrad_splits(rows, N, K, E);
    if (s > 1) w.sums = align16((size_t)s * E * N * K * 4);
    if (N % 8) w.pack_a = rows_n;
    if (K % 8) w.pack_b = rows_k;
  }
  return w;
}

static size_t pack_threads(int rows, int len) { return (size_t)rows * (pad8(len) / 8); }   // of one group

static hipError_t pack_rows(const uint16_t* src, size_t ld, size_t stride, int len, int rows, int groups, int src_rows,
                            const int32_t* row_index, int row_div, const int32_t* offsets, uint16_t* dst, hipStream_t s) {
  const int pad = pad8(len);
  const size_t n = pack_threads(rows, len);
  ProfScope prof("pack_rows", s);
  EXMOE_LAUNCH(prof, pack_rows_kernel, dim3((unsigned)((n + 255) / 256), groups), dim3(256), 0, s, src, ld, stride, len, rows,
               src_rows, row_index, row_div, offsets, dst, pad);
  return hipGetLastError();
}

template <class ET, int MODE, int BP, int BQ, int WP, int WQ, bool ALIGNED>
static hipError_t launch_rows(const GroupedArgs& a, const char* name, hipStream_t s) {
  const long long max_p = row_tiles(a.rows, a.E, BP);
  const int qt = ceil_div(MODE == kMM ? a.N : a.K, BQ);
  ProfScope prof(name, s);
  EXMOE_LAUNCH(prof, (grouped_kernel<ET, MODE, BP, BQ, WP, WQ, ALIGNED>), dim3((unsigned)(max_p * qt)),
               dim3(64 * WP * WQ), 0, s, a, 0, qt, 1);
  return hipGetLastError();
}

template <class ET, int MODE, int TP, int TQ, int WP, int WQ, int D, int OCC>
static hipError_t launch_wide(const GroupedArgs& a, const char* name, hipStream_t s) {
  constexpr int BP = 32 * TP * WP, BQ = 32 * TQ * WQ;
  const long long max_p = row_tiles(a.rows, a.E, BP);
  const int qt = ceil_div(MODE == kMM ? a.N : a.K, BQ);
  ProfScope prof(name, s);
  EXMOE_LAUNCH(prof, (grouped_wide_kernel<ET, MODE, TP, TQ, WP, WQ, D, OCC>), dim3((unsigned)(max_p * qt)),
               dim3(64 * WP * WQ), 0, s, a, 0, qt, 1);
  return hipGetLastError();
}

static bool op_aligned(const void* p, size_t ld, size_t stride, int len) {
  return aligned16(p) && ld % 8 == 0 && stride % 8 == 0 && len % 8 == 0;
}

// Whether an operand of n rows, ld apart, len long, can be addressed with 32-bit offsets.
static bool op_span(size_t n, size_t ld, int len) { return n == 0 || 2 * ((n - 1) * ld + len) < kMaxSpan; }
// The same where the n rows are the summed axis: a slice's rows past the end (up to 63) have
// to lie past the buffer too, not wrap around into it.
static bool sum_span(size_t n, size_t ld, int len) { return ld < kMaxSpan && op_span(n + 64, ld, len); }

// Rows of the tiles: 256 x 256 on 8 waves (one workgroup per compute unit) moves half the bytes
// per product of 128 x 128 on 4 waves (two per unit, so that one's start and end hide behind
// the other's loop). 320 x 256 keeps most experts in one tile where their rows scatter around a
// little less than 256 to 320: an expert of 257 rows costs two tiles of 256, which read its W
// twice. Measured on 64 experts of 2048 x 2048, rows per expert on average, evenly routed /
// skewed, us:
//         96          128         160         200         256         288    320    375
//   128   135 / 145   157 / 164   170 / 170   177 / 191   217 / 211
//   256   137 / 168   142 / 167   146 / 168   148 / 172   201 / 214   219    223    232
//   320                                       150 / 183   164 / 193   190    223    241
// The gradient of x, 200 rows: 208 / 165 / 173 on 128, 256, 320; 256 rows, skewed: 245 / 232 on
// 256, 320. From 512 rows on 256 and 320 are within 9% of each other, either way: 8 experts of
// 14336 x 4096 with 1024 rows each 1096 / 879 / 864 on 128, 256, 320; one of 8192 x 8192 846 / 924 on
// 256, 320.
// The large tiles need to give every compute unit one.
static int tile_rows(int rows, int Q, int E) {
  const int each = rows / E;
  if (each < 160 || (long long)(rows / 256) * ceil_div(Q, 256) < 256) return 128;
  return each > 256 * 9 / 10 && each <= 320 * 9 / 10 ? 320 : 256;
}

template <class ET, int TP, int TQ, int NW, int D, bool ALIGNED>
static hipError_t launch_narrow(const GroupedArgs& a, hipStream_t s) {
  const long long max_p = row_tiles(a.rows, a.E, 16 * TP);
  const int qt = ceil_div(a.N, 16 * TQ);
  ProfScope prof("grouped_mm", s);
  EXMOE_LAUNCH(prof, (grouped_narrow_kernel<ET, TP, TQ, NW, D, ALIGNED>), dim3((unsigned)(max_p * qt)), dim3(64 * NW), 0, s, a, qt);
  return hipGetLastError();
}

template <class ET, int TP, int NW>
static hipError_t launch_narrow_dgrad(const GroupedArgs& a, hipStream_t s) {
  const long long max_p = row_tiles(a.rows, a.E, 16 * TP);
  const int qt = ceil_div(a.K, 64);
  ProfScope prof("grouped_dgrad", s);
  EXMOE_LAUNCH(prof, (grouped_narrow_dgrad_kernel<ET, TP, NW>), dim3((unsigned)(max_p * qt)), dim3(64 * NW), 0, s, a, qt);
  return hipGetLastError();
}

// The gradient of x on 16-row blocks instead of 128 x 128 tiles when those leave compute units
// idle. Measured with 64 experts of 2048 x 2048, us: 1 token (8 rows, 128 tiles) 21 / 31,
// 4 tokens (512 tiles) 56 / 54, 16 tokens 96 / 95; 16 tokens, 8 experts of 2048 x 512 13 / 25.
static bool narrow_dgrad(const GroupedArgs& a) {
  return a.rows <= 10 * a.E && (long long)(a.E < a.rows ? a.E : a.rows) * ceil_div(a.K, 128) < 512 && op_span(16, a.lda, a.len_a);
}

// Rows per expert up to which the forward product runs on 16-row blocks (narrow) instead of
// 128-row tiles. Measured on 64 experts of 2048 x 2048, us: 2 rows per expert 83 / 117,
// 8 rows 97 / 128, 16 rows 127 / 130, 32 rows 182 / 131. Operands of any alignment, 13 experts
// of 517 x 1003: 10 rows 11 / 39, 39 rows 21 / 42, 60 rows 28 / 44, 630 rows 193 / 61. Skewed (Zipf),
// 2048 x 2048: 64 experts, 2 rows on average 67 / 99, 8 rows 102 / 123, 16 rows 127 / 130; 128 experts,
// 4 rows 146 / 155, 16 rows 246 / 196 (the largest expert's W is read once per 16 of its rows; the
// host knows the average alone).
// (Where 16 x 16 blocks are more than one launch holds, 128 x 128 tiles may still fit.)
constexpr int kNarrowRows = 16, kNarrowRowsAny = 128;

// Fewer 128 x 128 tiles than half the CUs: 64 x 64 blocks whose waves split the reduction (500
// rows, E = 4, N = 1024, K = 2048: 25.5 -> 14.7 us, the gradient of x of 1000 rows, N = 2048,
// K = 384 28.0 -> 18.6 us; with 154 and 207 tiles 21.3 -> 20.2 and 33.8 -> 37.7 us).
static bool few_tiles(int rows, int Q, int E) {
  return (rows / 128 + (long long)(E < rows ? E : rows)) * ceil_div(Q, 128) < 128;
}
// Of those, too few 64 x 64 blocks: 16-row blocks (blocks of 64 x 64, us on 64 x 64 / 16 rows:
// forward 18, K = 6496, 34 / 16; 38, K = 2176, 12.6 / 8.7; 56, K = 2048, 12.1 / 8.5; 96, K = 1024,
// 9.9 / 11.1; 176, K = 2048, 14.7 / 19.3; gradient of x 21, N = 4224, 27 / 16; 56, N = 2048, 14.8 /
// 11.1; 304, N = 512, 13.6 / 18.2).
static bool few_blocks(int rows, int Q, int E) {
  return (rows / 64 + (long long)(E < rows ? E : rows)) * ceil_div(Q, 64) < 80;
}

template <class ET>
static hipError_t mm_type(const GroupedArgs& a, hipStream_t s) {
  const bool al = op_aligned(a.a, a.lda, 0, a.len_a) && op_aligned(a.b, a.ldb, a.b_stride, a.len_b);
  if (!al) {
    if (a.rows <= kNarrowRowsAny * (long long)a.E && tiles_fit(a.rows, a.N, a.E, 16, 16, 512)) return launch_narrow<ET, 1, 1, 8, 64, false>(a, s);
    return launch_rows<ET, kMM, 128, 128, 2, 2, false>(a, "grouped_mm", s);
  }
  if (a.rows <= kNarrowRows * (long long)a.E && op_span(a.x_rows, a.lda, a.K) && op_span(16, a.ldb, a.K) &&
      tiles_fit(a.rows, a.N, a.E, 16, 16, 256))
    return launch_narrow<ET, 1, 1, 4, 64, true>(a, s);
  if (!op_span(a.x_rows, a.lda, a.len_a) || !op_span(a.N, a.ldb, a.len_b))
    return launch_rows<ET, kMM, 128, 128, 2, 2, true>(a, "grouped_mm", s);
  if (few_tiles(a.rows, a.N, a.E))
    return few_blocks(a.rows, a.N, a.E) ? launch_narrow<ET, 1, 1, 4, 64, true>(a, s) : launch_narrow<ET, 4, 4, 4, 32, true>(a, s);
  const int height = tile_rows(a.rows, a.N, a.E);
  if (height == 320) return launch_wide<ET, kMM, 5, 2, 2, 4, 64, 2>(a, "grouped_mm", s);
  if (height == 256) return launch_wide<ET, kMM, 4, 2, 2, 4, 64, 2>(a, "grouped_mm", s);
  return launch_wide<ET, kMM, 2, 2, 2, 2, 64, 2>(a, "grouped_mm", s);
}

// Copies the operands that need it; a then describes the copies.
static hipError_t pack_a_rows(GroupedArgs& a, int len, bool gather, hipStream_t s) {
  hipError_t e = pack_rows(a.a, a.lda, 0, len, a.rows, 1, gather ? a.x_rows : a.rows, gather ? a.row_index : nullptr,
                           a.row_div, nullptr, a.pack_a, s);
  a.a = a.pack_a;
  a.lda = a.len_a = pad8(len);
  return e;
}
static hipError_t pack_weights(GroupedArgs& a, hipStream_t s) {
  hipError_t e = pack_rows(a.b, a.ldb, a.b_stride, a.K, a.N, a.E, a.N, nullptr, 1, a.offsets, a.pack_b, s);
  a.b = a.pack_b;
  a.ldb = a.len_b = pad8(a.K);
  a.b_stride = (size_t)a.N * a.ldb;
  return e;
}

hipError_t launch_grouped_mm(const GroupedArgs& given, hipStream_t s) {
  GroupedArgs a = given;
  hipError_t e = hipSuccess;
  if (a.pack_a) {
    if ((e = pack_a_rows(a, a.K, true, s)) != hipSuccess) return e;
    a.x_rows = a.rows;
    a.row_index = nullptr;
    a.row_div = 1;
  }
  if (a.pack_b && (e = pack_weights(a, s)) != hipSuccess) return e;
  return a.fp16 ? mm_type<ElemFP16>(a, s) : mm_type<ElemBF16>(a, s);
}

template <class ET>
static hipError_t dgrad_type(const GroupedArgs& a, hipStream_t s) {
  const bool al = op_aligned(a.a, a.lda, 0, a.len_a) && op_aligned(a.b, a.ldb, a.b_stride, a.len_b);
  GroupedArgs r = a;
  if (a.flat_to_sorted) {
    r.out = a.ws;
    r.vec = a.K % 4 == 0;
    r.ldo = (size_t)a.K;
    r.out_f32 = 1;
  }
  hipError_t e;
  const int height = tile_rows(a.rows, a.K, a.E);
  if (!al) e = launch_rows<ET, kDG, 128, 128, 2, 2, false>(r, "grouped_dgrad", s);
  else if (!op_span(a.rows, a.lda, a.len_a) || !sum_span(a.N, a.ldb, a.len_b))
    e = launch_rows<ET, kDG, 128, 128, 2, 2, true>(r, "grouped_dgrad", s);
  else if (narrow_dgrad(a)) e = launch_narrow_dgrad<ET, 1, 8>(r, s);
  else if (few_tiles(a.rows, a.K, a.E))
    e = few_blocks(a.rows, a.K, a.E) ? launch_narrow_dgrad<ET, 1, 8>(r, s) : launch_narrow_dgrad<ET, 4, 4>(r, s);
  else if (height == 320) e = launch_wide<ET, kDG, 5, 2, 2, 4, 64, 2>(r, "grouped_dgrad", s);
  else if (height == 256) e = launch_wide<ET, kDG, 4, 2, 2, 4, 64, 2>(r, "grouped_dgrad", s);
  else e = launch_wide<ET, kDG, 2, 2, 2, 2, 64, 2>(r, "grouped_dgrad", s);
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

hipError_t launch_grouped_dgrad(const GroupedArgs& given, hipStream_t s) {
  GroupedArgs a = given;
  hipError_t e = hipSuccess;
  if (a.pack_a && (e = pack_a_rows(a, a.N, false, s)) != hipSuccess) return e;
  if (a.pack_b && (e = pack_weights(a, s)) != hipSuccess) return e;
  return a.fp16 ? dgrad_type<ElemFP16>(a, s) : dgrad_type<ElemBF16>(a, s);
}

template <int BP, int BQ, int THREADS, class F>
static hipError_t launch_weights(const GroupedArgs& a, hipStream_t s, int splits, F kernel) {
  const int pt = ceil_div(a.N, BP), qt = ceil_div(a.K, BQ);
  const long long grid = (long long)pt * qt * a.E * splits;
  ProfScope prof("grouped_wgrad", s);
  EXMOE_LAUNCH(prof, kernel, dim3((unsigned)grid), dim3(THREADS), 0, s, a, pt, qt, splits);
  return hipGetLastError();
}
template <class ET, int TP, int TQ, int WP, int WQ, int D, int OCC>
static hipError_t launch_weights_wide(const GroupedArgs& a, hipStream_t s, int splits) {
  return launch_weights<32 * TP * WP, 32 * TQ * WQ, 64 * WP * WQ>(a, s, splits, grouped_wide_kernel<ET, kWG, TP, TQ, WP, WQ, D, OCC>);
}

template <class ET>
static hipError_t wgrad_type(const GroupedArgs& a, hipStream_t s) {
  const int splits = wgrad_splits(a.rows, a.N, a.K, a.E);
  hipError_t e;
  if (!op_aligned(a.a, a.lda, 0, a.len_a) || !op_aligned(a.b, a.ldb, 0, a.len_b))
    e = launch_weights<128, 128, 256>(a, s, splits, grouped_kernel<ET, kWG, 128, 128, 2, 2, false>);
  else if (!sum_span(a.rows, a.lda, a.len_a) || !op_span(a.x_rows, a.ldb, a.len_b))
    e = launch_weights<128, 128, 256>(a, s, splits, grouped_kernel<ET, kWG, 128, 128, 2, 2, true>);
  else if (a.rows / a.E >= 768 && splits == 1 && (long long)a.E * ceil_div(a.N, 256) * ceil_div(a.K, 256) >= 256)
    e = launch_weights_wide<ET, 4, 2, 2, 4, 64, 2>(a, s, splits);
  else
    // few rows per output: 128 x 128 tiles with shallow slices, three workgroups per compute
    // unit, so that the stores of one run beside the loops of others (256 rows per expert of
    // 2048 x 2048: 289 us against 329 us on 256 x 256 tiles; 1024 rows of 14336 x 4096:
    // 1166 against 1103 us)
    e = launch_weights_wide<ET, 2, 2, 2, 2, 32, 3>(a, s, splits);
  if (e != hipSuccess || splits == 1) return e;
  const size_t n = (size_t)a.E * a.N * a.K;
  ProfScope prof("split_sum", s);
  if (a.K % 4 == 0)
    EXMOE_LAUNCH(prof, (split_sum_kernel<ET, 4>), dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, s, a.ws, splits, a.E,
                 a.N, a.K, a.out, a.ldo, a.o_stride, a.out_f32, a.vec);
  else
    EXMOE_LAUNCH(prof, (split_sum_kernel<ET, 1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.ws, splits, a.E,
                 a.N, a.K, a.out, a.ldo, a.o_stride, a.out_f32, a.vec);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedArgs& given, hipStream_t s) {
  GroupedArgs a = given;
  hipError_t e = hipSuccess;
  if (a.rows > 0 && a.pack_a && (e = pack_a_rows(a, a.N, false, s)) != hipSuccess) return e;
  if (a.rows > 0 && a.pack_b) {
    e = pack_rows(a.b, a.ldb, 0, a.K, a.rows, 1, a.x_rows, a.row_index, a.row_div, nullptr, a.pack_b, s);
    if (e != hipSuccess) return e;
    a.b = a.pack_b;
    a.ldb = a.len_b = pad8(a.K);
    a.x_rows = a.rows;
    a.row_index = nullptr;
    a.row_div = 1;
  }
  return a.fp16 ? wgrad_type<ElemFP16>(a, s) : wgrad_type<ElemBF16>(a, s);
}

// Whether each launch of a call holds its threads: the copies, the products' last resort (128 x
// 128 tiles, and 256 x 256 on twice the threads) and the sums. Checked before anything runs.
static bool call_fits(int op, int rows, int N, int K, int E, int k, const GroupedWorkspace& need) {
  const size_t most = (size_t)kMaxThreads;
  if (op == EXMOE_GROUPED_WGRAD) {
    const long long wide = (long long)E * ceil_div(N, 256) * ceil_div(K, 256) * 512,
                    tiles = (long long)E * ceil_div(N, 128) * ceil_div(K, 128) * wgrad_splits(rows, N, K, E) * 256;
    return wide <= kMaxThreads && tiles <= kMaxThreads && (!need.pack_a || pack_threads(rows, N) <= most) &&
           (!need.pack_b || pack_threads(rows, K) <= most);
  }
  const int Q = op == EXMOE_GROUPED_MM ? N : K;
  if (!tiles_fit(rows, Q, E, 128, 128, 256) || !tiles_fit(rows, Q, E, 256, 256, 512)) return false;
  if (need.pack_a && pack_threads(rows, op == EXMOE_GROUPED_MM ? K : N) > most) return false;
  if (need.pack_b && pack_threads(N, K) > most) return false;
  return k == 0 || (size_t)(rows / k) * (K % 4 == 0 ? K / 4 : K) <= most;
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

static int check_size(bool fits, const char* what) {
  return fits ? EXMOE_OK : set_error(EXMOE_ERR_UNSUPPORTED, "%s: more output tiles or copied elements than one launch holds", what);
}

static void set_workspace(GroupedArgs& a, const GroupedWorkspace& need, void* ws) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.ws = reinterpret_cast<float*>(p);
  a.pack_a = need.pack_a ? reinterpret_cast<uint16_t*>(p + need.sums) : nullptr;
  a.pack_b = need.pack_b ? reinterpret_cast<uint16_t*>(p + need.sums + need.pack_a) : nullptr;
}

extern "C" size_t exmoe_grouped_mm_workspace_bytes(int op, int rows, int N, int K, int E, int k) {
  if (op < EXMOE_GROUPED_MM || op > EXMOE_GROUPED_WGRAD || k < 0) {
    set_error(EXMOE_ERR_INVALID_ARGUMENT, "unknown grouped operator %d or negative k %d", op, k);
    return 0;
  }
  if (grouped_shape(rows, N, K, E, EXMOE_DTYPE_BF16, EXMOE_DTYPE_BF16)) return 0;
  return grouped_workspace(op, rows, N, K, E, k).total();
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
  const GroupedWorkspace need = grouped_workspace(EXMOE_GROUPED_MM, rows, N, K, E, 0);
  EXMOE_TRY(check_size(call_fits(EXMOE_GROUPED_MM, rows, N, K, E, 0, need), "exmoe_grouped_mm"));
  EXMOE_TRY(check_ws(need.total(), workspace, ws_bytes));
  const MemRows mx = mem_matrix("x", x, row_index ? x_rows : rows, ldx, K, 2), mw = mem_matrices("w", w, E, w_stride, N, ldw, K, 2),
                mi = mem_flat("row_index", row_index, (size_t)rows * 4), mo = mem_flat("expert_offsets", expert_offsets, (E + 1) * 4),
                my = mem_matrix("y", y, rows, ldy, N, ob);
  EXMOE_TRY(check_apart(my, {mx, mw, mi, mo}));
  EXMOE_TRY(check_apart(mem_flat("workspace", workspace, need.total()), {mx, mw, mi, mo, my}));
  GroupedArgs a{};
  a.a = static_cast<const uint16_t*>(x); a.b = static_cast<const uint16_t*>(w); a.lda = ldx; a.ldb = ldw;
  a.b_stride = E > 1 ? w_stride : 0; a.offsets = expert_offsets; a.row_index = row_index; a.row_div = row_div; a.x_rows = x_rows;
  a.rows = rows; a.N = N; a.K = K; a.E = E; a.out = y; a.ldo = ldy; a.fp16 = dtype == EXMOE_DTYPE_FP16;
  a.out_f32 = ob == 4; a.vec = vec_store(y, ldy, 0, a.out_f32); a.len_a = a.len_b = K;
  set_workspace(a, need, workspace);
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
  const GroupedWorkspace need = grouped_workspace(EXMOE_GROUPED_DGRAD, rows, N, K, E, flat_to_sorted ? k : 0);
  EXMOE_TRY(check_size(call_fits(EXMOE_GROUPED_DGRAD, rows, N, K, E, flat_to_sorted ? k : 0, need), "exmoe_grouped_mm_dgrad"));
  EXMOE_TRY(check_ws(need.total(), workspace, ws_bytes));
  const MemRows md = mem_matrix("dy", dy, rows, lddy, N, 2), mw = mem_matrices("w", w, E, w_stride, N, ldw, K, 2),
                mi = mem_flat("flat_to_sorted", flat_to_sorted, (size_t)rows * 4),
                mo = mem_flat("expert_offsets", expert_offsets, (E + 1) * 4),
                mx = mem_matrix("dx", dx, flat_to_sorted ? rows / k : rows, lddx, K, ob);
  EXMOE_TRY(check_apart(mx, {md, mw, mi, mo}));
  EXMOE_TRY(check_apart(mem_flat("workspace", workspace, need.total()), {md, mw, mi, mo, mx}));
  GroupedArgs a{};
  a.a = static_cast<const uint16_t*>(dy); a.b = static_cast<const uint16_t*>(w); a.lda = lddy; a.ldb = ldw;
  a.b_stride = E > 1 ? w_stride : 0; a.offsets = expert_offsets; a.row_div = 1; a.x_rows = rows; a.rows = rows; a.N = N; a.K = K;
  a.E = E; a.out = dx; a.ldo = lddx; a.fp16 = dtype == EXMOE_DTYPE_FP16; a.out_f32 = ob == 4;
  a.vec = vec_store(dx, lddx, 0, a.out_f32); a.flat_to_sorted = flat_to_sorted; a.k = k; a.len_a = N;
  a.len_b = K;
  set_workspace(a, need, workspace);
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
  const GroupedWorkspace need = grouped_workspace(EXMOE_GROUPED_WGRAD, rows, N, K, E, 0);
  EXMOE_TRY(check_size(call_fits(EXMOE_GROUPED_WGRAD, rows, N, K, E, 0, need), "exmoe_grouped_mm_wgrad"));
  EXMOE_TRY(check_ws(need.total(), workspace, ws_bytes));
  const MemRows md = mem_matrix("dy", dy, rows, lddy, N, 2), mx = mem_matrix("x", x, rows == 0 ? 0 : row_index ? x_rows : rows, ldx, K, 2),
                mi = mem_flat("row_index", row_index, (size_t)rows * 4), mo = mem_flat("expert_offsets", expert_offsets, (E + 1) * 4),
                mw = mem_matrices("dw", dw, E, dw_stride, N, lddw, K, ob);
  EXMOE_TRY(check_apart(mw, {md, mx, mi, mo}));
  EXMOE_TRY(check_apart(mem_flat("workspace", workspace, need.total()), {md, mx, mi, mo, mw}));
  GroupedArgs a{};
  a.a = static_cast<const uint16_t*>(dy); a.b = static_cast<const uint16_t*>(x); a.lda = lddy; a.ldb = ldx;
  a.offsets = expert_offsets; a.row_index = row_index; a.row_div = row_div; a.x_rows = x_rows; a.rows = rows; a.N = N;
  a.K = K; a.E = E; a.out = dw; a.ldo = lddw; a.o_stride = E > 1 ? dw_stride : 0; a.fp16 = dtype == EXMOE_DTYPE_FP16;
  a.out_f32 = ob == 4; a.vec = vec_store(dw, lddw, a.o_stride, a.out_f32); a.len_a = N; a.len_b = K;
  set_workspace(a, need, workspace);
  return launched(launch_grouped_wgrad(a, stream), "exmoe_grouped_mm_wgrad");
}
