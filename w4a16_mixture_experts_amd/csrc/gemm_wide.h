// The pipelined tile loop of the matrix products (grouped.hip, lora.hip): aligned 16-bit
// operands of any length on v_mfma_f32_32x32x16, fp32 accumulation, gfx950.
#pragma once

#include "gemm_tile.h"

namespace exmoe {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(ElemBF16, bf16x8 a, bf16x8 b, f32x16 c) {
  typedef __bf16 b8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(ElemFP16, bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// s_waitcnt vmcnt(N) alone
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }
// Barrier that memory operations do not move across (it does not wait for them itself).
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---- operands of the pipelined tile loop: 32-row and 32-column fragments for
// v_mfma_f32_32x32x16 (lane l: row or column l % 32, summed positions 8 (l / 32) + 0..7; D:
// column l % 32, rows 8 (r / 4) + 4 (l / 32) + r % 4 of register r). The copies are buffer
// loads into LDS: an offset past the buffer's end writes zeros, so rows past a segment,
// columns past a matrix and positions past the summed axis cost no memory traffic and need
// no selects in the loop. A lane's offsets inside the slice are fixed; the slice moves by the
// scalar offset. Offsets have 32 bits: an operand must span less than kMaxSpan bytes.
constexpr uint32_t kMaxSpan = 0x80000000u;
constexpr uint32_t kNowhere = 0xC0000000u;   // past the end of any operand

typedef __amdgpu_buffer_rsrc_t buf_t;
__device__ __forceinline__ buf_t make_buf(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)bytes, 0x00027000);
}
__device__ __forceinline__ void buf_copy16(buf_t r, void* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}

// Rows (summed axis contiguous), B of them, D deep. The 16-byte chunk c of row i lies at
// position c ^ swz(i): the 16 rows of a fragment read cover all 64 banks once.
template <int B, int NW, int D>
struct WideRows {
  static constexpr int kChunks = D / 8, kRows = 64 / kChunks, kSlots = B / (kRows * NW);
  static constexpr int kReads = 1;   // LDS reads of a fragment
  static_assert(B % (kRows * NW) == 0 && (D == 32 || (D == 64 && NW % 2 == 0)), "rows per slice");
  buf_t buf;
  int red, wave, chunk;              // chunk: the lane's first summed position in a slice
  uint32_t voff[kSlots];

  static __device__ __forceinline__ int swz(int row) { return D == 64 ? (row >> 1) & 7 : (row >> 2) & 3; }
  // row_off(i): byte offset of row i of the tile, or kNowhere for zeros
  template <class F>
  __device__ __forceinline__ void init(buf_t b, int red_, int wave_, int lane, F row_off) {
    buf = b;
    red = red_;
    wave = wave_;
    chunk = 8 * ((lane % kChunks) ^ swz(wave * kRows + lane / kChunks));   // the same in each of the lane's rows
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      const uint32_t o = row_off((i * NW + wave) * kRows + lane / kChunks);
      voff[i] = o == kNowhere ? o : o + 2 * chunk;
    }
  }
  // positions past the summed axis are zeros (a slice wholly past it moves nothing)
  __device__ __forceinline__ void stage(uint16_t* lds, int k0) const {
    const bool in = k0 + chunk < red;
    const uint32_t soff = k0 < red ? 2 * (uint32_t)k0 : 0;   // never past the buffer's end
#pragma unroll
    for (int i = 0; i < kSlots; i++) buf_copy16(buf, lds + (i * NW + wave) * kRows * D, in ? voff[i] : kNowhere, soff);
  }
  // rows r0..r0+31, summed positions 16 ks + 8 (lane / 32) + 0..7 of the slice
  static __device__ __forceinline__ bf16x8 frag(const uint16_t* lds, int r0, int ks, int lane) {
    const int row = r0 + (lane & 31);
    return *reinterpret_cast<const bf16x8*>(lds + row * D + 8 * ((2 * ks + (lane >> 5)) ^ swz(row)));
  }
};

// Columns (summed axis outermost), B of them, D deep. The 32-byte unit u of row r lies at
// position u ^ 2 (r & 3): 32 lanes of a transposing read touch two adjacent units of four
// rows, which then cover all 64 banks once.
template <int B, int NW, int D>
struct WideCols {
  static constexpr int kChunks = B / 8, kRows = 64 / kChunks, kSlots = D / (kRows * NW);
  static constexpr int kReads = 2;
  static_assert(B >= 128 && B <= 512 && D % (kRows * NW) == 0, "columns per slice");
  buf_t buf;
  uint32_t ld2;              // bytes per row of the summed axis
  int red, wave, lane;
  uint32_t voff[kSlots];

  __device__ __forceinline__ int slot_row(int i) const { return (i * NW + wave) * kRows + lane / kChunks; }
  // ncols: columns of the matrix from the tile's first one on; GATHER: the offsets of a
  // slice's rows are given with it (stage_rows)
  template <bool GATHER>
  __device__ __forceinline__ void init(buf_t b, uint32_t ld2_, int red_, int ncols, int wave_, int lane_) {
    buf = b;
    ld2 = ld2_;
    red = red_;
    wave = wave_;
    lane = lane_;
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      const int row = slot_row(i), pos = lane % kChunks;
      const uint32_t c = 32 * ((pos >> 1) ^ (2 * (row & 3))) + 16 * (pos & 1);
      voff[i] = c < 2 * (uint32_t)ncols ? c + (GATHER ? 0 : (uint32_t)row * ld2) : kNowhere;
    }
  }
  // rows past the summed axis lie past the buffer's end (a slice wholly past it moves nothing)
  __device__ __forceinline__ void stage(uint16_t* lds, int k0) const {
    const bool in = k0 < red;
    const uint32_t soff = in ? (uint32_t)k0 * ld2 : 0;
#pragma unroll
    for (int i = 0; i < kSlots; i++) buf_copy16(buf, lds + (i * NW + wave) * kRows * B, in ? voff[i] : kNowhere, soff);
  }
  // rows: byte offsets of the slice's rows, or kNowhere, in LDS
  __device__ __forceinline__ void stage_rows(uint16_t* lds, const uint32_t* rows) const {
    uint32_t r[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; i++) r[i] = rows[slot_row(i)];
#pragma unroll
    for (int i = 0; i < kSlots; i++)
      buf_copy16(buf, lds + (i * NW + wave) * kRows * B,
                 r[i] == kNowhere || voff[i] == kNowhere ? kNowhere : r[i] + voff[i], 0);
  }
  // columns c0..c0+31, summed positions 16 ks + 8 (lane / 32) + 0..7: two transposing reads,
  // each turning 4 rows x 16 columns per 16 lanes into 4 consecutive rows of a column per lane
  static __device__ __forceinline__ bf16x8 frag(const uint16_t* lds, int c0, int ks, int lane) {
    const int r3 = (lane >> 2) & 3, row = 16 * ks + 8 * (lane >> 5) + r3;
    const uint16_t* p = lds + row * B + 16 * (((c0 >> 4) + ((lane >> 4) & 1)) ^ (2 * r3)) + 4 * (lane & 3);
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * B));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// ---- few rows: each wave copies its own slices of both operands into its own part of LDS
// (no barrier), two D-deep slices in flight, and the waves split the summed axis slice by
// slice. Straight loads in fragment order touch a different row in each of four neighbouring
// lanes, which costs a vector memory unit four times the cycles of a copy of whole 128- or
// 256-byte row pieces (64 tokens beside W 2048 x 2048 and their adapters: 16.5 -> 9.7 us).
template <int B, int D>
struct NarrowRows {
  static constexpr int kChunks = D / 8, kRows = 64 / kChunks, kSlots = B / kRows, kElems = B * D;
  static_assert((D == 32 || D == 64) && B % 16 == 0, "rows of a slice");
  buf_t buf;
  int red, c0;               // c0: the lane's chunk in its first row
  uint32_t voff[kSlots];

  static __device__ __forceinline__ int swz(int row) { return D == 64 ? (row >> 1) & 7 : (row >> 2) & 3; }
  // row_off(i): byte offset of row i, or kNowhere for zeros
  template <class F>
  __device__ __forceinline__ void init(buf_t b, int red_, int lane, F row_off) {
    buf = b;
    red = red_;
    c0 = (lane % kChunks) ^ swz(lane / kChunks);
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      const uint32_t o = row_off(i * kRows + lane / kChunks);
      voff[i] = o == kNowhere ? o : o + 16 * chunk(i);
    }
  }
  __device__ __forceinline__ int chunk(int i) const { return c0 ^ swz(i * kRows); }   // (row bits of i and of the lane are apart)
  // positions past the summed axis are zeros (a slice wholly past it moves nothing)
  __device__ __forceinline__ void stage(uint16_t* lds, int k0) const {
    const uint32_t soff = k0 < red ? 2 * (uint32_t)k0 : 0;
#pragma unroll
    for (int i = 0; i < kSlots; i++)
      buf_copy16(buf, lds + i * kRows * D, k0 + 8 * chunk(i) < red ? voff[i] : kNowhere, soff);
  }
  // rows r0..r0 + 15, positions 32 kk + 8 (lane / 16) + 0..7 of the slice
  static __device__ __forceinline__ bf16x8 frag(const uint16_t* lds, int r0, int kk, int lane) {
    const int row = r0 + (lane & 15);
    return *reinterpret_cast<const bf16x8*>(lds + row * D + 8 * ((4 * kk + (lane >> 4)) ^ swz(row)));
  }
};

// 64 columns of an operand whose summed axis is outermost, D rows of it a slice. The 32-byte
// unit u of row r lies at position u ^ f(r): the eight rows that 32 lanes of a transposing
// read touch cover all 64 banks once.
template <int D>
struct NarrowCols {
  static constexpr int kSlots = D / 8, kElems = 64 * D;
  static_assert(D % 16 == 0, "rows of a slice");
  buf_t buf;
  uint32_t ld2;              // bytes per row of the summed axis
  int red;
  uint32_t voff[kSlots];

  static __device__ __forceinline__ int f(int row) { return ((row >> 1) & 1) | (((row >> 3) & 1) << 1); }
  __device__ __forceinline__ void init(buf_t b, uint32_t ld2_, int red_, int ncols, int lane) {
    buf = b;
    ld2 = ld2_;
    red = red_;
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      const int row = 8 * i + (lane >> 3), pos = lane & 7;
      const uint32_t c = 32 * ((pos >> 1) ^ f(row)) + 16 * (pos & 1);
      voff[i] = c < 2 * (uint32_t)ncols ? c + (uint32_t)row * ld2 : kNowhere;
    }
  }
  // rows past the summed axis lie past the buffer's end (a slice wholly past it moves nothing)
  __device__ __forceinline__ void stage(uint16_t* lds, int k0) const {
    const bool in = k0 < red;
    const uint32_t soff = in ? (uint32_t)k0 * ld2 : 0;
#pragma unroll
    for (int i = 0; i < kSlots; i++) buf_copy16(buf, lds + 512 * i, in ? voff[i] : kNowhere, soff);
  }
  // columns c0..c0 + 15, positions 32 kk + 8 (lane / 16) + 0..7 of the slice
  static __device__ __forceinline__ bf16x8 frag(const uint16_t* lds, int c0, int kk, int lane) {
    const int row = 32 * kk + 8 * (lane >> 4) + ((lane >> 2) & 3);   // and row + 4: the same f
    const uint16_t* p = lds + 64 * row + 16 * ((c0 >> 4) ^ f(row)) + 4 * (lane & 3);
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 64));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// acc[j][i] += block j of w (16 columns of the output) times rows 16 i.. of x, over this
// wave's slices; s_a, s_b: this wave's two parts of LDS, OpX::kElems + OpW::kElems each.
template <class ET, int TP, int TQ, int NW, int D, class OpX, class OpW>
__device__ __forceinline__ void narrow_product(const OpX& x, const OpW& w, int red, int wave, int lane, uint16_t* s_a,
                                               uint16_t* s_b, f32x4 (&acc)[TQ][TP]) {
  constexpr int kCopies = OpX::kSlots + OpW::kSlots;
  auto issue = [&](int s, uint16_t* lds) __attribute__((always_inline)) {
    const int k0 = (s * NW + wave) * D;
    w.stage(lds, k0);
    x.stage(lds + OpW::kElems, k0);
  };
  auto compute = [&](const uint16_t* lds) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < D / 32; kk++) {
      bf16x8 fw[TQ], fx[TP];
#pragma unroll
      for (int j = 0; j < TQ; j++) fw[j] = OpW::frag(lds, 16 * j, kk, lane);
#pragma unroll
      for (int i = 0; i < TP; i++) fx[i] = OpX::frag(lds + OpW::kElems, 16 * i, kk, lane);
#pragma unroll
      for (int j = 0; j < TQ; j++)
#pragma unroll
        for (int i = 0; i < TP; i++) acc[j][i] = ET::mfma(fw[j], fx[i], acc[j][i]);
    }
    wait_lds();   // read, before the next copies into this part
    asm volatile("" ::: "memory");
  };
  const int n = (red + D * NW - 1) / (D * NW);
  issue(0, s_a);
  issue(1, s_b);
  for (int s = 0; s < n; s += 2) {
    wait_vm<kCopies>();
    asm volatile("" ::: "memory");
    compute(s_a);
    issue(s + 2, s_a);
    wait_vm<kCopies>();
    asm volatile("" ::: "memory");
    compute(s_b);
    issue(s + 3, s_b);
  }
  wait_vm<0>();   // no copy is left behind
}

// Where a tile's outputs go: element base + row ld + q of ptr.
struct TileOut {
  void* ptr;
  size_t base, ld;
  bool f32, vec;   // vec: rows can be stored 16 bytes at a time
};

// One tile: rows p0.. (those below plim exist), columns q0.. (below Q) of the output, summed
// over red positions. WP x WQ waves of TP x TQ blocks of 32 x 32.
// Two D-deep slices in LDS, each D / 16 steps; a step's fragments are read while the step
// before runs on MFMA (two register sets), the reads and copies spread between the MFMAs.
// The slice's one barrier comes before its first reads: the wave then still holds the
// fragments of the last step of the slice before, so every wave is done reading that slice
// and the next one is copied into its buffer right there, with a whole slice's time to land.
// Row blocks are dealt to the WP wave rows in turn, and blocks past plim are skipped: a
// ragged tile costs the MFMAs of its rows, spread over all waves.
// GATHER (columns form of Q): load_row(r) loads what leads to row r of Q's source, and
// row_bytes(value) makes its byte offset (or kNowhere); both for r < red only.
// adjust(i, p, acc): changes the sums of row block i (lane's row p) before they are stored;
// out_row(p): row of the output.
// An output's whole sum (of its part, where a gradient of W is split) is one chain of MFMAs in an
// fp32 accumulator: relative error against 64 bits over 8192 summed positions 5.7e-7 (mixed signs)
// and 4.7e-7 (all positive), 65536 rows of a gradient of W 1.2e-6 and 7e-7; the installed BLAS in
// fp32 9.5e-7, 1.3e-6, 3.5e-6 and 4.5e-6.
// 256 x 256 tiles (4, 2, 2, 4, 64): 8192 x 8192 x 8192 bf16 in 829 us, 1.33 PFLOP/s; MFMA
// busy 80% of the cycles at the about 1.5 GHz that the chip sustains under it, the rest is
// waiting for copies at the barrier. Slices half as deep in four buffers: 909 us (twice the
// barriers); four waves of 128 x 128: 922 us (nothing hides a lone wave's barrier); the lines of
// the slice after next asked for into L2 a slice ahead: 876 us.
template <class ET, int TP, int TQ, int WP, int WQ, int D, bool GATHER, class OpP, class OpQ, class LoadRow,
          class RowBytes, class Adjust, class OutRow>
__device__ __forceinline__ void wide_tile(const OpP& op_p, const OpQ& op_q, int red, int p0, int plim, int q0, int Q,
                                          const TileOut& out, LoadRow load_row, RowBytes row_bytes, Adjust adjust,
                                          OutRow out_row) {
  constexpr int NW = WP * WQ, BP = 32 * TP * WP, BQ = 32 * TQ * WQ;
  // (separate arrays: the compiler then sees that reading one does not wait for copies into another)
  __shared__ __attribute__((aligned(16))) uint16_t s_p0[BP * D], s_p1[BP * D], s_q0[BQ * D], s_q1[BQ * D];
  // GATHER: byte offsets of the rows of Q, two chunks of slices
  constexpr int kIdxSlices = 8, kIdx = kIdxSlices * D;
  __shared__ uint32_t s_row[GATHER ? 2 * kIdx : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave / WQ, wq = wave % WQ;

  // chunk c of the rows' offsets goes to LDS a slice before its first use; what leads to
  // them is loaded a chunk ahead
  constexpr int kMine = GATHER ? (kIdx + 64 * NW - 1) / (64 * NW) : 1;
  int crow[kMine];
  auto load_chunk = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int r = c * kIdx + tid + i * 64 * NW;
      crow[i] = r < red ? load_row(r) : -1;
    }
  };
  auto store_chunk = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int r = tid + i * 64 * NW;
      if (kIdx % (64 * NW) == 0 || r < kIdx) s_row[(c & 1) * kIdx + r] = crow[i] < 0 ? kNowhere : row_bytes(crow[i]);
    }
  };
  auto stage = [&](int s, uint16_t* lp, uint16_t* lq) __attribute__((always_inline)) {
    op_p.stage(lp, s * D);
    if constexpr (GATHER) op_q.stage_rows(lq, s_row + (s & (2 * kIdxSlices - 1)) * D);
    else op_q.stage(lq, s * D);
  };

  f32x16 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; j++)
#pragma unroll
    for (int i = 0; i < TP; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[j][i][r] = 0.f;

  const int steps = (red + D - 1) / D;
  auto block_p = [&](int i) __attribute__((always_inline)) { return 32 * (i * WP + wp); };   // first row of row block i
  int nblk = 0;                                                                              // of them hold rows
#pragma unroll
  for (int i = 0; i < TP; i++) nblk += p0 + block_p(i) < plim ? 1 : 0;
  nblk = __builtin_amdgcn_readfirstlane(nblk);

  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  bf16x8 fp[2][TP], fq[2][TQ];
  auto read = [&](auto set_c, const uint16_t* lp, const uint16_t* lq, int ks) __attribute__((always_inline)) {
    constexpr int set = decltype(set_c)::value;
#pragma unroll
    for (int j = 0; j < TQ; j++) fq[set][j] = OpQ::frag(lq, (wq * TQ + j) * 32, ks, lane);
#pragma unroll
    for (int i = 0; i < TP; i++) fp[set][i] = OpP::frag(lp, block_p(i), ks, lane);
  };
  auto multiply = [&](auto full, auto set_c) __attribute__((always_inline)) {
    constexpr int set = decltype(set_c)::value;
#pragma unroll
    for (int i = 0; i < TP; i++) {
      if (decltype(full)::value || i < nblk) {
#pragma unroll
        for (int j = 0; j < TQ; j++) acc[j][i] = mfma32(ET{}, fq[set][j], fp[set][i], acc[j][i]);
      }
    }
  };
  // spreads a step's reads (and copies) between its MFMAs
  constexpr int kReads = OpP::kReads * TP + OpQ::kReads * TQ, kMfma = TP * TQ;
  auto interleave = [&](auto full, auto copies_c) __attribute__((always_inline)) {
    if constexpr (decltype(full)::value) {
      constexpr int copies = decltype(copies_c)::value;
#pragma unroll
      for (int i = 0; i < kMfma; i++) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        const int nr = (i + 1) * kReads / kMfma - i * kReads / kMfma;
        if (nr == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (nr == 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        const int nc = (i + 1) * copies / kMfma - i * copies / kMfma;
        if (nc == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        if (nc == 2) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
      }
    }
  };
  using None = std::integral_constant<int, 0>;
  // slice s in (cp, cq), slice s + 1 (or zeros past the last one) copied into (np, nq)
  auto slice = [&](auto full, int s, uint16_t* cp, uint16_t* cq, uint16_t* np, uint16_t* nq)
      __attribute__((always_inline)) {
    wait_lds();      // this wave holds its last fragments of slice s - 1
    wait_vm<0>();    // its copies of slice s have landed
    block_barrier();
    read(S0{}, cp, cq, 0);
    stage(s + 1, np, nq);
    multiply(full, S1{});
    interleave(full, std::integral_constant<int, OpP::kSlots + OpQ::kSlots>{});
    read(S1{}, cp, cq, 1);
    multiply(full, S0{});
    interleave(full, None{});
#pragma unroll
    for (int ks = 2; ks < D / 16; ks += 2) {
      read(S0{}, cp, cq, ks);
      multiply(full, S1{});
      interleave(full, None{});
      read(S1{}, cp, cq, ks + 1);
      multiply(full, S0{});
      interleave(full, None{});
    }
    if constexpr (GATHER) {
      if ((s & (kIdxSlices - 1)) == kIdxSlices - 2) {
        store_chunk(s / kIdxSlices + 1);
        load_chunk(s / kIdxSlices + 2);
      }
    }
  };
  auto loop = [&](auto full) __attribute__((always_inline)) {
    for (int s = 0; s < steps; s += 2) {
      slice(full, s, s_p0, s_q0, s_p1, s_q1);
      if (s + 1 < steps) slice(full, s + 1, s_p1, s_q1, s_p0, s_q0);
    }
    multiply(full, S1{});
  };
  if (steps > 0) {
    if constexpr (GATHER) {
      load_chunk(0);
      store_chunk(0);
      load_chunk(1);
      __syncthreads();
    }
    stage(0, s_p0, s_q0);
    const bf16x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < TQ; j++) fq[1][j] = zero;
#pragma unroll
    for (int i = 0; i < TP; i++) fp[1][i] = zero;
    if (nblk == TP) loop(std::true_type{});
    else loop(std::false_type{});
    wait_vm<0>();    // no copy is left behind the workgroup's end
  }

  // Lane l holds p = l % 32 and q = 8 g + 4 (l / 32) + 0..3 (registers 4 g..4 g + 3) of a block:
  // each wave turns a row block at a time through its own part of LDS, so that a row leaves
  // in pieces of 16 bytes a lane, 32 TQ outputs together (16-byte chunks swizzled by the row,
  // so that 16 rows of a write hit distinct banks). The stores bypass the caches: a gradient of
  // W of 1 GiB left in 289 us instead of 485 us (2048 tokens, 64 experts of 2048 x 2048, fp32).
#pragma unroll
  for (int i = 0; i < TP; i++)
    if (i < nblk) adjust(i, p0 + block_p(i) + (lane & 31), acc);
  constexpr int kCols = 32 * TQ;
  block_barrier();   // everyone is done with the slices
  uint16_t* mine = wave % 4 == 0 ? s_p0 : wave % 4 == 1 ? s_p1 : wave % 4 == 2 ? s_q0 : s_q1;
  static_assert(NW == 4 || NW == 8, "one part of the slices' LDS per wave");
  static_assert(32 * kCols * 4 <= (BP < BQ ? BP : BQ) * D * 2 / (NW / 4), "a block of fp32 rows fits");
  if (NW == 8 && wave >= 4) mine += (BP < BQ ? BP : BQ) * D / 2;
  const int qw = q0 + wq * kCols;
  auto flush = [&](auto f32_c) __attribute__((always_inline)) {
    constexpr bool F32 = decltype(f32_c)::value;
    constexpr int SZ = F32 ? 4 : 2, kPitch = kCols * SZ;
    constexpr int kLanes = kCols * SZ / 16, kRows = 64 / kLanes;   // lanes (16-byte chunks) per row, rows per store
    auto at = [&](int row, int byte) __attribute__((always_inline)) {
      const int swz = kLanes >= 16 ? row & 15 : kLanes == 8 ? (row >> 1) & 7 : (row >> 2) & 3;
      return reinterpret_cast<char*>(mine) + row * kPitch + (byte ^ (16 * swz));
    };
#pragma unroll
    for (int i = 0; i < TP; i++) {
      if (i >= nblk) break;
#pragma unroll
      for (int j = 0; j < TQ; j++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
          const f32x16& c = acc[j][i];
          char* p = at(lane & 31, (32 * j + 8 * g + 4 * (lane >> 5)) * SZ);
          if constexpr (F32)
            *reinterpret_cast<f32x4*>(p) = f32x4{c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
          else
            *reinterpret_cast<uint2*>(p) = make_uint2(ET::pack2(c[4 * g], c[4 * g + 1]), ET::pack2(c[4 * g + 2], c[4 * g + 3]));
        }
      const int pb = p0 + block_p(i);
      if (!out.vec) {   // (uniform) rows that start anywhere: neighbouring lanes write neighbouring elements
#pragma unroll 2
        for (int e = 0; e < 32 * kCols / 64; e++) {   // (unrolled further, its addresses push sums out of the registers)
          const int row = (64 * e + lane) / kCols, col = (64 * e + lane) % kCols, q = qw + col;
          if (pb + row < plim && q < Q) {
            const size_t o = out.base + (size_t)out_row(pb + row) * out.ld + q;
            if constexpr (F32) static_cast<uint32_t*>(out.ptr)[o] = *reinterpret_cast<const uint32_t*>(at(row, col * SZ));
            else static_cast<uint16_t*>(out.ptr)[o] = *reinterpret_cast<const uint16_t*>(at(row, col * SZ));
          }
        }
        continue;
      }
#pragma unroll
      for (int r = 0; r < 32; r += kRows) {
        const int row = r + lane / kLanes, col = (lane % kLanes) * (16 / SZ), q = qw + col;
        const uint4 v = *reinterpret_cast<const uint4*>(at(row, col * SZ));
        if (pb + row < plim && q < Q) {
          char* dst = static_cast<char*>(out.ptr) + (out.base + (size_t)out_row(pb + row) * out.ld + q) * SZ;
          if (q + 16 / SZ <= Q) {
            __builtin_nontemporal_store(__builtin_bit_cast(i32x4, v), reinterpret_cast<i32x4*>(dst));
          } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 16 / SZ; e++)
              if (q + e < Q) {
                if constexpr (F32) reinterpret_cast<uint32_t*>(dst)[e] = w[e];
                else reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
              }
          }
        }
      }
    }
  };
  if (out.f32) flush(std::true_type{});
  else flush(std::false_type{});
}

}  // namespace exmoe
