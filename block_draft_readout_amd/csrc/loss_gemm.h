// The matrix products of the vocabulary losses (gfx950): logits, and the
// gradients that come back through them.
//
//   C[m, n] = sum_k A(m, k) B(n, k), fp32 accumulation, with either operand
//   stored with the reduction index fast (rows of k: hidden states, weights as
//   the logits read them) or slow (columns of k: weights as d hidden reads
//   them, d logits and hidden states as d weight reads them).  Both directions
//   read the tensors as they lie in memory; nothing is transposed in HBM.
//
// A workgroup of WM x WN waves owns a tile of C, a wave WTM x WTN MFMA tiles of
// 16 x 16.  The reduction advances 128 bytes per operand row and step (64 bf16
// or 32 fp32 elements); a step's slices are copied global -> LDS by
// buffer-to-LDS loads into a ring of STAGES stages, one workgroup barrier per
// step.
//  * reduction fast: an LDS row is one operand row's 128 bytes, its eight
//    16-byte chunks XOR-permuted by the row; an MFMA operand is one 16-byte read.
//  * reduction slow: an LDS row is one k with the tile's columns side by side;
//    an MFMA operand of bf16 is two transposing reads (ds_read_b64_tr_b16: 16
//    lanes read 4 k x 16 columns, lane i receives column i's four values), of
//    fp32 four 4-byte reads.  The 32-byte units of a bf16 LDS row are
//    XOR-permuted by k so the 16 pieces of one read fall on distinct banks.
// Loads place the permuted data by choosing which bytes each lane fetches.
//
// Everything past a tensor's edge reads as zero: rows and slow-k slices end
// with the buffer descriptor, a fast-k tail is cut per lane.  The number of
// rows that take part is a device value (rows without a target are compacted
// away before the products run), so grids are sized for all rows and
// workgroups past the last live tile leave at once.
#pragma once

#include "train_device.h"

namespace bdr {

enum LossEpilogue {
  LE_STATS,     // per row and tile: running maximum and sum of exp of the scaled logits
  LE_DLOGITS,   // coef (softmax - onehot), rounded to the storage type
  LE_PARTIAL,   // fp32, one slab per reduction split, stored or added to
  LE_OUT        // rounded to the storage type
};

// One stretch of the reduction: operand bases, row strides (elements) and extent.
// d logits, operand a of every gradient product (those with slow b), lie in
// panels of 128 bytes: element (m, v) at a + v / KB * lda + m * KB + v % KB with
// KB elements in 128 bytes and lda from panel to panel.  A step's slice is then
// contiguous, where rows of the vocabulary's length would put each of its 128
// byte pieces into another memory page.
struct LossSeg {
  const void* a;
  const void* b;
  int64_t lda, ldb;
  int64_t k;
};

// rows whose labels a wave of a weight gradient holds
constexpr int kHeldRows = 512;

struct LossGemm {
  LossSeg seg[2];          // the second one with the reduction fast on both sides only
  const int32_t* live;     // device: rows that take part
  int64_t M, N;            // extents of C (M: an upper bound where live_m)
  int live_m, live_k;      // the row count is *live / the first segment's extent is *live
  int tiles_n;
  int band;                // tile rows per band of the tile order
  int splits;              // reduction splits (LE_PARTIAL)
  int two;                 // 1: row m of d logits is the sum of rows 2 m and 2 m + 1 as stored (0: row m)
  // logits epilogues
  float scale2;            // log2(e) / temperature
  const int32_t* label;    // [M] target entry or NULL (LE_OUT: of the reduction's rows)
  int label0;              // vocabulary entry of column 0
  float2* stat;            // [M, tiles_n] (maximum, sum) in units of log2
  float* picked;           // [M] logit of the label
  float* resid;            // [M] what rounding d logits left at the label, or NULL (LE_OUT: added, up to
                           // kHeldRows rows)
  const float* lse2;       // [M] log2 of the softmax denominator
  const float* lse_corr;   // [M] fp32: factor of the probabilities, what rounding lse2 left
  const float* coef;       // [M] gradient factor
  void* out;               // LE_DLOGITS panels, LE_PARTIAL [splits, slab], LE_OUT [M, ldo]
  int64_t ldo;             // LE_DLOGITS: N padded to whole panels
  int64_t slab;            // elements of a split, or of a panel
  int accumulate;          // LE_PARTIAL: add to what is there
};

template <typename S_, bool AKS_, bool BKS_, int WM_, int WN_, int WTM_, int WTN_, int STAGES_,
          bool LOOP_ = false, bool NT_B_ = false, int STAGES_A_ = STAGES_, int JOIN_ = 0>
struct LossTile {
  using S = S_;
  static constexpr bool AKS = AKS_, BKS = BKS_;   // reduction slow
  static constexpr int WM = WM_, WN = WN_, WTM = WTM_, WTN = WTN_, STAGES = STAGES_;
  static constexpr bool LOOP = LOOP_;             // a workgroup walks several tiles
  static constexpr bool NT_B = NT_B_;             // B is streamed once: non-temporal loads
  static constexpr int STAGES_A = STAGES_A_;      // stages of A where it has fewer (it comes from L2)
  // Steps whose products are summed by themselves before they join the running sum (0: a chain
  // of MFMAs on the running sum).  An eighth of the roundings at its size, for as many registers
  // again: in fp32 a step (8 MFMAs), in bf16 four (8), where the tile has them.
  static constexpr int JOIN = sizeof(S) == 4 ? 1 : JOIN_;
  static constexpr int WAVES = WM * WN;
  static constexpr int BM = 16 * WM * WTM, BN = 16 * WN * WTN;
  static constexpr int KB = 128 / static_cast<int>(sizeof(S));
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr bool STAGED = WTM * WTN <= 32;
  static constexpr int RING_BYTES = STAGES_A * A_BYTES + STAGES * B_BYTES;
  // a stage's A and B lie side by side, or in rings of their own
  static constexpr int LAG = STAGES - STAGES_A;   // steps by which A's loads trail B's
  static constexpr int A_STEP = LAG ? A_BYTES : A_BYTES + B_BYTES;
  static constexpr int B_STEP = LAG ? B_BYTES : A_BYTES + B_BYTES;
  static constexpr int B_BASE = LAG ? STAGES_A * A_BYTES : A_BYTES;
  // scratch of the epilogues: row statistics, or a wave's 16 output rows.  A
  // workgroup with more tiles to come keeps it beside the ring.
  static constexpr int OUT_ROW = 16 * WTN * static_cast<int>(sizeof(S));
  // 16 bytes between the rows: the 16 rows a store instruction reaches then start in
  // 16 different groups of four banks (an odd multiple of 16 bytes, over 256)
  static constexpr int OUT_PITCH = OUT_ROW + 16;
  static constexpr int SCRATCH = std::max(WN * BM * 8, WAVES * 16 * OUT_PITCH);
  static constexpr int LDS_BYTES = LOOP ? RING_BYTES + SCRATCH : std::max(RING_BYTES, SCRATCH);
  static constexpr int PER_CU = 160 * 1024 / LDS_BYTES;   // workgroups a compute unit holds
  // may meet d logits in two terms, which only few rows have (they take no larger tiles)
  static constexpr bool TWO = sizeof(S) == 2 && BM <= 128;
  // waves of a SIMD to leave registers for: the workgroups LDS has room for, up to two
  // waves (without it 128 x 128 d logits took 268 registers, so one workgroup of two
  // ran: 4258 us instead of 2260, 4096 rows of 5120, 20 x 2560 entries)
  static constexpr int SIMD_WAVES = std::max(1, std::min(2, PER_CU * WAVES / 4));
  static constexpr int LOADS_A = BM / 8 / WAVES, LOADS_B = BN / 8 / WAVES;
  static constexpr int LOADS = LOADS_A + LOADS_B;
  // LDS reads the compiler schedules, per half step (the transposing ones are its own block)
  static constexpr int SLOW_READS = sizeof(S) == 2 ? 0 : 4;
  static constexpr int READS = WTM * (AKS ? SLOW_READS : 1) + WTN * (BKS ? SLOW_READS : 1);
  static constexpr int MFMAS = WTM * WTN * Elem<S>::MFMA_PER16;   // per half step
  static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "loads split evenly over the waves");
  static_assert((!AKS || BM % 64 == 0) && (!BKS || BN % 64 == 0), "slow rows are multiples of 128 bytes");
  static_assert(LAG == 0 || (STAGES_A == 2 && !LOOP), "A in two stages, B in more");
  static_assert(PER_CU >= 1, "tile fits");
};

// XOR of the 32-byte unit index in a reduction-slow bf16 LDS row of ROWB bytes.
// A transposing read takes 16 pieces of 32 bytes, rows {8 g + j : g, j < 4} (or
// those plus 4), in two passes of 32 lanes (g = 0, 1, then 2, 3) over 64 banks:
// (row * ROWB + unit * 32) mod 256 has to differ between the 8 rows of a pass.
template <int ROWB>
__device__ __forceinline__ uint32_t slow_swizzle(uint32_t kr) {
  const uint32_t g = (kr >> 3) & 1u, j = kr & 3u;
  return ROWB % 256 == 0 ? (j << 1) | g : (j >> 1) | (g << 1);
}

// 16 bytes per lane, global -> LDS: lane l's land at dst + 16 l (dst uniform)
template <int AUX>
__device__ __forceinline__ void load_lds16(rsrc_t r, uint32_t off, char* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, off,
                                           0, 0, AUX);
}

// Transposing reads of NA operand tiles whose 8-byte pieces this lane names at
// LDS addresses ad[0 .. NA), and of NB more at ad[NA ..): four 16-bit values of
// column lane % 16 from 4 k rows, and from the 4 k rows after those (RA / RB bytes
// per k row), HALF k rows into the stage.  One block of assembly with its own wait: the
// compiler takes the intrinsic for a possible write to LDS and waits for every
// buffer-to-LDS load in flight before it, which costs the loads' latency once a
// step (d weight of 12 x 2560 entries, 4096 rows of 5120, 256 x 320 tiles: 1530 ->
// 1090 us).
#define BDR_TR_READ(i, o0, o1)                                                          \
  "ds_read_b64_tr_b16 %[l" #i "], %[a" #i "] offset:%c[" #o0 "]\n\t"                     \
  "ds_read_b64_tr_b16 %[h" #i "], %[a" #i "] offset:%c[" #o1 "]\n\t"
#define BDR_TR_OUT(i) [l##i] "=&v"(l[i]), [h##i] "=&v"(h[i])
#define BDR_TR_IN(i) [a##i] "v"(ad[i])
#define BDR_TR_4(m, i0, i1, i2, i3, ...) \
  m(i0, ##__VA_ARGS__) m(i1, ##__VA_ARGS__) m(i2, ##__VA_ARGS__) m(i3, ##__VA_ARGS__)
#define BDR_TR_IMM                                                                       \
  [p0] "n"(HALF * RA), [p1] "n"((HALF + 4) * RA), [q0] "n"(HALF * RB), [q1] "n"((HALF + 4) * RB)
template <int NA, int RA, int NB, int RB, int HALF>
__device__ __forceinline__ void lds_read_tr(const uint32_t (&ad)[NA + NB], u32x4_t (&f)[NA + NB]) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  u32x2_t l[NA + NB], h[NA + NB];
  if constexpr (NA == 2 && NB == 0) {
    asm volatile(BDR_TR_READ(0, p0, p1) BDR_TR_READ(1, p0, p1) "s_waitcnt lgkmcnt(0)"
                 : BDR_TR_OUT(0), BDR_TR_OUT(1)
                 : BDR_TR_IN(0), BDR_TR_IN(1), BDR_TR_IMM
                 : "memory");
  } else if constexpr (NA == 4 && NB == 0) {
    asm volatile(BDR_TR_4(BDR_TR_READ, 0, 1, 2, 3, p0, p1) "s_waitcnt lgkmcnt(0)"
                 : BDR_TR_OUT(0), BDR_TR_OUT(1), BDR_TR_OUT(2), BDR_TR_OUT(3)
                 : BDR_TR_IN(0), BDR_TR_IN(1), BDR_TR_IN(2), BDR_TR_IN(3), BDR_TR_IMM
                 : "memory");
  } else if constexpr (NA == 5 && NB == 0) {
    asm volatile(BDR_TR_4(BDR_TR_READ, 0, 1, 2, 3, p0, p1) BDR_TR_READ(4, p0, p1)
                 "s_waitcnt lgkmcnt(0)"
                 : BDR_TR_OUT(0), BDR_TR_OUT(1), BDR_TR_OUT(2), BDR_TR_OUT(3), BDR_TR_OUT(4)
                 : BDR_TR_IN(0), BDR_TR_IN(1), BDR_TR_IN(2), BDR_TR_IN(3), BDR_TR_IN(4), BDR_TR_IMM
                 : "memory");
  } else if constexpr (NA == 4 && NB == 2) {
    asm volatile(BDR_TR_READ(4, q0, q1) BDR_TR_READ(5, q0, q1)
                 BDR_TR_4(BDR_TR_READ, 0, 1, 2, 3, p0, p1) "s_waitcnt lgkmcnt(0)"
                 : BDR_TR_OUT(0), BDR_TR_OUT(1), BDR_TR_OUT(2), BDR_TR_OUT(3), BDR_TR_OUT(4),
                   BDR_TR_OUT(5)
                 : BDR_TR_IN(0), BDR_TR_IN(1), BDR_TR_IN(2), BDR_TR_IN(3), BDR_TR_IN(4),
                   BDR_TR_IN(5), BDR_TR_IMM
                 : "memory");
  } else if constexpr (NA == 4 && NB == 5) {
    asm volatile(BDR_TR_4(BDR_TR_READ, 4, 5, 6, 7, q0, q1) BDR_TR_READ(8, q0, q1)
                 BDR_TR_4(BDR_TR_READ, 0, 1, 2, 3, p0, p1) "s_waitcnt lgkmcnt(0)"
                 : BDR_TR_OUT(0), BDR_TR_OUT(1), BDR_TR_OUT(2), BDR_TR_OUT(3), BDR_TR_OUT(4),
                   BDR_TR_OUT(5), BDR_TR_OUT(6), BDR_TR_OUT(7), BDR_TR_OUT(8)
                 : BDR_TR_IN(0), BDR_TR_IN(1), BDR_TR_IN(2), BDR_TR_IN(3), BDR_TR_IN(4),
                   BDR_TR_IN(5), BDR_TR_IN(6), BDR_TR_IN(7), BDR_TR_IN(8), BDR_TR_IMM
                 : "memory");
  } else if constexpr (NA == 8 && NB == 5) {
    asm volatile(BDR_TR_4(BDR_TR_READ, 8, 9, 10, 11, q0, q1) BDR_TR_READ(12, q0, q1)
                 BDR_TR_4(BDR_TR_READ, 0, 1, 2, 3, p0, p1) BDR_TR_4(BDR_TR_READ, 4, 5, 6, 7, p0, p1)
                 "s_waitcnt lgkmcnt(0)"
                 : BDR_TR_OUT(0), BDR_TR_OUT(1), BDR_TR_OUT(2), BDR_TR_OUT(3), BDR_TR_OUT(4),
                   BDR_TR_OUT(5), BDR_TR_OUT(6), BDR_TR_OUT(7), BDR_TR_OUT(8), BDR_TR_OUT(9),
                   BDR_TR_OUT(10), BDR_TR_OUT(11), BDR_TR_OUT(12)
                 : BDR_TR_IN(0), BDR_TR_IN(1), BDR_TR_IN(2), BDR_TR_IN(3), BDR_TR_IN(4),
                   BDR_TR_IN(5), BDR_TR_IN(6), BDR_TR_IN(7), BDR_TR_IN(8), BDR_TR_IN(9),
                   BDR_TR_IN(10), BDR_TR_IN(11), BDR_TR_IN(12), BDR_TR_IMM
                 : "memory");
  } else {
    static_assert(NA < 0, "no transposing read of this shape");
  }
#pragma unroll
  for (int i = 0; i < NA + NB; ++i) f[i] = u32x4_t{l[i].x, l[i].y, h[i].x, h[i].y};
}

// 32-bit LDS address of a pointer into the workgroup's LDS
__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p));
}

// Joins two running (maximum, sum of 2^(x - maximum)) pairs.
__device__ __forceinline__ float2 merge_stat(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float ref = m == -INFINITY ? 0.f : m;
  return float2{m, a.y * __builtin_amdgcn_exp2f(a.x - ref) + b.y * __builtin_amdgcn_exp2f(b.x - ref)};
}

__device__ __forceinline__ void store4(uint16_t* p, f32x4_t v) {
  *reinterpret_cast<uint2*>(p) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}
__device__ __forceinline__ void store4(float* p, f32x4_t v) { *reinterpret_cast<f32x4_t*>(p) = v; }

__device__ __forceinline__ f32x4_t load4(const uint16_t* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return f32x4_t{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                 __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u)};
}
__device__ __forceinline__ f32x4_t load4(const float* p) {
  return *reinterpret_cast<const f32x4_t*>(p);
}

// what rounding x to bf16 leaves (nothing of an infinity)
__device__ __forceinline__ float left_over(float x) {
  const float hi = bf16_to_f32(rounded<uint16_t>(x));
  return fabsf(hi) == INFINITY ? 0.f : x - hi;
}

// Workgroup `block` of `blocks` (a multiple of 8) of one product.
template <typename T, int EPI>
__device__ __forceinline__ void loss_gemm_body(const LossGemm& g, int block, int blocks) {
  using S = typename T::S;
  constexpr int ES = static_cast<int>(sizeof(S));
  __shared__ __attribute__((aligned(16))) char lds[T::LDS_BYTES];
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int r16 = lane & 15;
  const int grp = lane >> 4;
  const int wm = wave % T::WM;
  const int wn = wave / T::WM;

  // Tiles of this workgroup: each XCD takes a contiguous run of the work items, its
  // workgroups one each or every wgs-th of the run, so those at work together share
  // slices in that XCD's L2.
  const int two = T::TWO ? g.two : 0;
  const int live = *g.live << (EPI == LE_PARTIAL || EPI == LE_OUT ? two : 0);   // rows as stored
  const int64_t M = g.live_m ? live : g.M;
  const int tiles_m = static_cast<int>((M + T::BM - 1) / T::BM);
  const int tiles = tiles_m * g.tiles_n;
  // work items: the tiles of the first reduction split, of the second, ...
  const int items = EPI == LE_PARTIAL ? tiles * g.splits : tiles;
  const int per_xcd = (items + 7) / 8;
  const int wgs = blocks / 8;
  const int xcd = block % 8, in_xcd = block / 8;   // workgroup b runs on XCD b % 8
  if (in_xcd >= per_xcd) return;   // whole workgroup
  const int item = xcd * per_xcd + in_xcd;
  if (item >= items) return;
  const int split = EPI == LE_PARTIAL ? item / tiles : 0;
  const int t_first = item - split * tiles;
  const int t_end = T::LOOP ? min(tiles, (xcd + 1) * per_xcd) : t_first + 1;
  auto tile_at = [&](int t, int& tm, int& tn) {
    const int band = t / (g.band * g.tiles_n);
    const int bh = min(g.band, tiles_m - g.band * band);
    const int bidx = t - g.band * g.tiles_n * band;
    tm = g.band * band + bidx % bh;
    tn = bidx / bh;
  };

  constexpr bool kTwo = !T::AKS && !T::BKS;   // two segments may be given
  // reduction steps of this workgroup: the first segment's, then the second's
  const int64_t k0 = g.live_k ? live : g.seg[0].k;
  const int steps0 = static_cast<int>((k0 + T::KB - 1) / T::KB);
  const int total = steps0 + (kTwo ? static_cast<int>((g.seg[1].k + T::KB - 1) / T::KB) : 0);
  int s_lo = 0, s_hi = total;
  if constexpr (EPI == LE_PARTIAL) {
    s_lo = static_cast<int>(static_cast<int64_t>(total) * split / g.splits);
    s_hi = static_cast<int>(static_cast<int64_t>(total) * (split + 1) / g.splits);
  }

  const int s_data = s_hi;        // steps from here on read zeros
  s_hi = max(s_hi, s_lo + 1);     // nothing to reduce: one step of zeros

  // per-lane offsets of this wave's loads
  const uint32_t lrow = static_cast<uint32_t>(lane >> 3);
  const uint32_t lchunk = (static_cast<uint32_t>(lane) & 7u) ^ lrow;
  // byte offset of load q's chunk of this lane inside the step's slice of an
  // operand with row stride ld (panels: with ld from panel to panel)
  // (two rows of A's reduction to one of B's where d logits come in two terms)
  auto lane_off = [&](auto slow, auto rowbytes, auto panels, int q, uint32_t ld,
                      int two = 0) -> uint32_t {
    const uint32_t i = static_cast<uint32_t>(wave + T::WAVES * q);
    if constexpr (!decltype(slow)::value) {
      return (8u * i + lrow) * (decltype(panels)::value ? 128u : ld * ES) + lchunk * 16u;
    } else {
      constexpr uint32_t ROWB = decltype(rowbytes)::value;
      const uint32_t o = i * 1024u + static_cast<uint32_t>(lane) * 16u;
      const uint32_t kr = o / ROWB;
      uint32_t p = o % ROWB;
      if constexpr (ES == 2) p = (((p >> 5) ^ slow_swizzle<ROWB>(kr)) << 5) | (p & 16u);
      if constexpr (decltype(panels)::value) return (p >> 7) * ld * ES + kr * 128u + (p & 127u);
      return (kr >> two) * ld * ES + p;
    }
  };
  typedef std::integral_constant<bool, T::AKS> ASlow;
  typedef std::integral_constant<bool, T::BKS> BSlow;
  typedef std::integral_constant<uint32_t, T::BM * ES> ARow;
  typedef std::integral_constant<uint32_t, T::BN * ES> BRow;

  // the gradient products have one segment: their loads' offsets never change
  constexpr bool kPanels = T::BKS;
  typedef std::integral_constant<bool, kPanels> APanels;
  const int two_b = EPI == LE_OUT ? two : 0;
  uint32_t off_a[T::LOADS_A], off_b[T::LOADS_B];
  if constexpr (kPanels) {
    static_for<T::LOADS_A>([&](auto q) {
      off_a[q] = lane_off(ASlow{}, ARow{}, APanels{}, q, static_cast<uint32_t>(g.seg[0].lda));
    });
    static_for<T::LOADS_B>([&](auto q) {
      off_b[q] = lane_off(BSlow{}, BRow{}, std::false_type{}, q, static_cast<uint32_t>(g.seg[0].ldb),
                          two_b);
    });
  }
  // slow panels: LDS row of this lane in load 0, and how many rows further each
  // load is (rows past the reduction's end are cut per lane)
  constexpr uint32_t kLoadRows = T::WAVES * 1024u / (T::BM * ES);
  const uint32_t kr0 = (static_cast<uint32_t>(wave) * 1024u + static_cast<uint32_t>(lane) * 16u) / (T::BM * ES);
  static_assert(!T::AKS || T::WAVES * 1024 % (T::BM * ES) == 0, "loads step by whole rows");

  // The loads run STAGES - 1 steps ahead of the MFMAs, with LOOP from one tile's
  // last step straight into the next tile's first, so a tile's epilogue overlaps
  // them.  Past the last tile they read zeros (empty descriptors), so that every step
  // issues the same loads and the waits count alike.
  int ld_t = t_first, ld_s = s_lo;   // tile and step of the next loads
  int64_t ld_m0 = 0, ld_n0 = 0;
  auto ld_tile = [&] {
    int tm, tn;
    tile_at(ld_t, tm, tn);
    ld_m0 = static_cast<int64_t>(tm) * T::BM;
    ld_n0 = static_cast<int64_t>(tn) * T::BN;
  };
  ld_tile();
  rsrc_t ra, rb;
  uint32_t ld_a = 0, ld_b = 0;
  uint32_t cut_a = 0, cut_b = 0;          // kOOB in the lanes past a fast-k tail
  uint32_t ld_rows = 0;                   // slow panels: k rows of the step
  char *dst_a = lds, *dst_b = lds;
  // Step `s` of the reduction: its segment, its first k there and how many are left
  // (none past the end).
  auto at_step = [&](int s, const LossSeg*& sg, int64_t& kk, int64_t& krem) {
    const bool second = kTwo && s >= steps0;
    sg = second ? &g.seg[1] : &g.seg[0];
    kk = static_cast<int64_t>(second ? s - steps0 : s) * T::KB;
    krem = (second ? sg->k : k0) - kk;
    if (s >= s_data || (T::LOOP && ld_t >= t_end)) krem = 0;
  };
  // descriptors of B's step ld_s into stage buf_b and A's LAG steps before it into buf_a
  auto dma_prep = [&](int buf_a, int buf_b) {
    const LossSeg *sb, *sa;
    int64_t kb, kb_rem, ka, ka_rem;
    at_step(ld_s, sb, kb, kb_rem);
    if constexpr (T::LAG > 0) {
      at_step(ld_s - T::LAG, sa, ka, ka_rem);
    } else {
      sa = sb;
      ka = kb;
      ka_rem = kb_rem;
    }
    ld_a = static_cast<uint32_t>(sa->lda);
    ld_b = static_cast<uint32_t>(sb->ldb);
    cut_a = static_cast<int64_t>(lchunk) * Elem<S>::PER16 < ka_rem ? 0u : kOOB;
    cut_b = static_cast<int64_t>(lchunk) * Elem<S>::PER16 < kb_rem ? 0u : kOOB;
    const int64_t krows = min<int64_t>(T::KB, kb_rem);
    const char* pa = static_cast<const char*>(sa->a);
    const char* pb = static_cast<const char*>(sb->b);
    uint32_t na, nb;
    if constexpr (T::AKS) {
      const int64_t left = min<int64_t>(T::BM / T::KB, (M + T::KB - 1) / T::KB - ld_m0 / T::KB);
      pa += (ld_m0 / T::KB * sa->lda + ka * T::KB) * ES;
      na = static_cast<uint32_t>((left * sa->lda - ka * T::KB) * ES);
      ld_rows = static_cast<uint32_t>(min<int64_t>(T::KB, ka_rem));
    } else if constexpr (kPanels) {
      pa += (ka / T::KB * sa->lda + ld_m0 * T::KB) * ES;
      na = static_cast<uint32_t>(min<int64_t>(T::BM, M - ld_m0) * 128);
    } else {
      pa += (ld_m0 * sa->lda + ka) * ES;
      na = static_cast<uint32_t>((min<int64_t>(T::BM, M - ld_m0) * sa->lda - ka) * ES);
    }
    if constexpr (T::BKS) {
      pb += ((kb >> two_b) * sb->ldb + ld_n0) * ES;
      nb = static_cast<uint32_t>(((krows >> two_b) * sb->ldb - ld_n0) * ES);
    } else {
      pb += (ld_n0 * sb->ldb + kb) * ES;
      nb = static_cast<uint32_t>((min<int64_t>(T::BN, g.N - ld_n0) * sb->ldb - kb) * ES);
    }
    ra = make_rsrc(pa, ka_rem > 0 ? na : 0u);
    rb = make_rsrc(pb, kb_rem > 0 ? nb : 0u);
    dst_a = lds + buf_a * T::A_STEP;
    dst_b = lds + T::B_BASE + buf_b * T::B_STEP;
    ++ld_s;
    if constexpr (T::LOOP) {
      if (ld_s == s_hi) {
        ld_s = s_lo;
        ld_t += wgs;
        if (ld_t < t_end) ld_tile();
      }
    }
  };
  auto dma_one = [&](auto qc) {
    constexpr int q = decltype(qc)::value;
    if constexpr (q < T::LOADS_A) {
      uint32_t off;
      if constexpr (T::AKS)
        off = kr0 + q * kLoadRows < ld_rows ? off_a[q] : kOOB;
      else if constexpr (kPanels)
        off = off_a[q];   // a panel's columns past the reduction's end are zeros
      else
        off = lane_off(ASlow{}, ARow{}, APanels{}, q, ld_a) | cut_a;
      load_lds16<0>(ra, off, dst_a + (wave + T::WAVES * q) * 1024);
    } else {
      constexpr int p = q - T::LOADS_A;
      const uint32_t off =
          T::BKS ? off_b[p] : lane_off(BSlow{}, BRow{}, std::false_type{}, p, ld_b) | cut_b;
      load_lds16<T::NT_B ? 2 : 0>(rb, off, dst_b + (wave + T::WAVES * p) * 1024);
    }
  };

  f32x4_t acc[T::WTM][T::WTN];
  f32x4_t part[T::WTM][T::WTN];   // JOIN: what has not joined acc
  auto& sum = [&]() -> auto& {
    if constexpr (T::JOIN > 0) return part; else return acc;
  }();
  typedef u32x4_t FragA[T::WTM];
  typedef u32x4_t FragB[T::WTN];
  // operand of MFMA tile `tile` (16 rows of the operand) in half `half` of a step
  auto read_op = [&](auto slow, auto rowbytes, const char* base, int tile, int half) -> u32x4_t {
    if constexpr (!decltype(slow)::value) {
      const uint32_t c = (static_cast<uint32_t>(4 * half + grp) ^ static_cast<uint32_t>(lane & 7)) * 16u;
      return *reinterpret_cast<const u32x4_t*>(base + static_cast<uint32_t>(tile * 16 + r16) * 128u + c);
    } else {
      constexpr uint32_t ROWB = decltype(rowbytes)::value;
      const char* p = base + static_cast<uint32_t>(16 * half + 4 * grp) * ROWB +
                      static_cast<uint32_t>(tile * 16 + r16) * 4u;
      u32x4_t v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint32_t*>(p + e * ROWB);
      return v;
    }
  };
  // LDS address of this lane's piece of slow bf16 tile `tile` at k row 0 of a stage
  auto slow_at = [&](auto rowbytes, int operand, int tile) -> uint32_t {
    constexpr uint32_t ROWB = decltype(rowbytes)::value;
    const uint32_t kr = static_cast<uint32_t>(8 * grp + (r16 >> 2));
    return lds_address(lds) + static_cast<uint32_t>(operand) + kr * ROWB +
           ((static_cast<uint32_t>(tile) ^ slow_swizzle<ROWB>(kr)) << 5) +
           static_cast<uint32_t>(lane & 3) * 8u;
  };
  uint32_t at_a[T::WTM], at_b[T::WTN];
  if constexpr (ES == 2 && T::AKS)
    static_for<T::WTM>([&](auto i) { at_a[i] = slow_at(ARow{}, 0, wm * T::WTM + decltype(i)::value); });
  if constexpr (ES == 2 && T::BKS)
    static_for<T::WTN>([&](auto j) {
      at_b[j] = slow_at(BRow{}, T::B_BASE, wn * T::WTN + decltype(j)::value);
    });
  auto read_frags = [&](int buf_a, int buf_b, auto halfc, FragA& a, FragB& b) {
    constexpr int half = decltype(halfc)::value;
    const uint32_t stage_a = static_cast<uint32_t>(buf_a * T::A_STEP);
    const uint32_t stage_b = static_cast<uint32_t>(buf_b * T::B_STEP);
    constexpr bool tr_a = ES == 2 && T::AKS, tr_b = ES == 2 && T::BKS;
    if constexpr (!tr_a)
      static_for<T::WTM>([&](auto i) {
        a[i] = read_op(ASlow{}, ARow{}, lds + stage_a, wm * T::WTM + decltype(i)::value, half);
      });
    if constexpr (!tr_b)
      static_for<T::WTN>([&](auto j) {
        b[j] = read_op(BSlow{}, BRow{}, lds + T::B_BASE + stage_b, wn * T::WTN + decltype(j)::value, half);
      });
    if constexpr (tr_a && tr_b) {
      uint32_t ad[T::WTM + T::WTN];
      u32x4_t f[T::WTM + T::WTN];
      static_for<T::WTM>([&](auto i) { ad[i] = at_a[i] + stage_a; });
      static_for<T::WTN>([&](auto j) { ad[T::WTM + j] = at_b[j] + stage_b; });
      lds_read_tr<T::WTM, T::BM * 2, T::WTN, T::BN * 2, 32 * half>(ad, f);
      static_for<T::WTM>([&](auto i) { a[i] = f[i]; });
      static_for<T::WTN>([&](auto j) { b[j] = f[T::WTM + j]; });
    } else if constexpr (tr_b) {
      uint32_t ad[T::WTN];
      static_for<T::WTN>([&](auto j) { ad[j] = at_b[j] + stage_b; });
      lds_read_tr<T::WTN, T::BN * 2, 0, 0, 32 * half>(ad, b);
    }
  };

  // the rows' labels stay in registers (a load in a tile's epilogue would wait for the
  // next tile's operands, which are on their way before it)
  constexpr int kHeld = EPI == LE_OUT && T::TWO ? kHeldRows / 64 : 1;
  int held[kHeld];
  if constexpr (EPI == LE_OUT && T::TWO) {
    static_for<kHeld>([&](auto c) {
      const int p = 64 * decltype(c)::value + lane;
      held[c] = g.resid && p < live ? g.label[p] : -1;
      asm volatile("" : "+v"(held[c]));   // loaded from here on
    });
  }

  // Per step: wait for its loads, one barrier, then per half the operand reads
  // and the MFMAs; the loads of step s + STAGES - 1 are spread over the first
  // half's MFMAs (all before them where there are fewer MFMAs than loads).
  static_for<T::STAGES - 1>([&](auto c) {
    constexpr int step_a = decltype(c)::value - T::LAG;   // A's: nothing before its first
    dma_prep(step_a < 0 ? 0 : step_a, decltype(c)::value);
    static_for<T::LOADS>([&](auto q) {
      if constexpr (decltype(q)::value >= T::LOADS_A || step_a >= 0) dma_one(q);
    });
  });
  dma_prep(T::STAGES_A - 1, T::STAGES - 1);
  constexpr int NT = T::WTM * T::WTN;
  constexpr bool kSpread = NT >= T::LOADS;
  // loads younger than a step's own when it begins: those of the STAGES - 2 steps after
  // it; with LAG B's of the step before, which that step issued after this step's A
  constexpr int kAhead = T::LAG ? T::LOADS_B : (T::STAGES - 2) * T::LOADS;
  // stores of an epilogue that are younger than the loads the next tile's first
  // step waits for (memory operations complete in order)
  constexpr int kStores = T::LOOP && (EPI == LE_DLOGITS || EPI == LE_OUT)
                              ? T::WTM * ((16 * T::OUT_ROW + 1023) / 1024) : 0;
  static_assert(!T::LOOP || T::STAGED, "an unstaged epilogue's stores are not counted");
  static_assert(kAhead + kStores < 64, "waits can count these");
  FragA a;
  FragB b;
  int buf = 0, buf_a = 0;   // stages of B and A
  for (int t = t_first; t < t_end; t += wgs) {
    static_for<T::WTM>([&](auto i) {
      static_for<T::WTN>([&](auto j) { acc[i][j] = part[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f}; });
    });
    for (int s = s_lo; s < s_hi; ++s) {
      // this wave's loads of the step have landed when at most those of the
      // STAGES - 2 steps after it remain; after the barrier every wave's have,
      // and every wave is done with the stage the next loads overwrite
      if (kStores > 0 && s == s_lo && t != t_first)
        BDR_WAIT_VM_LGKM(kAhead + kStores, 0);
      else
        BDR_WAIT_VM_LGKM(kAhead, 0);
      BDR_WG_BARRIER();
      if constexpr (!kSpread) static_for<T::LOADS>([&](auto q) { dma_one(q); });
      read_frags(buf_a, buf, std::integral_constant<int, 0>{}, a, b);
      static_for<NT>([&](auto ec) {
        constexpr int e = decltype(ec)::value;
        constexpr int every = kSpread ? NT / T::LOADS : NT;
        sum[e / T::WTN][e % T::WTN] =
            mma16(b[e % T::WTN], a[e / T::WTN], sum[e / T::WTN][e % T::WTN], S());
        if constexpr (kSpread && e % every == every - 1 && e / every < T::LOADS)
          dma_one(std::integral_constant<int, e / every>{});
      });
      read_frags(buf_a, buf, std::integral_constant<int, 1>{}, a, b);
      static_for<NT>([&](auto ec) {
        constexpr int e = decltype(ec)::value;
        sum[e / T::WTN][e % T::WTN] =
            mma16(b[e % T::WTN], a[e / T::WTN], sum[e / T::WTN][e % T::WTN], S());
      });
      if constexpr (kSpread) {   // keep that order through scheduling
        constexpr int every = NT / T::LOADS * Elem<S>::MFMA_PER16;
        if constexpr (T::READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, T::READS, 0);
        static_for<T::LOADS>([&](auto) {
          __builtin_amdgcn_sched_group_barrier(0x008, every, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        });
        if constexpr (T::MFMAS - every * T::LOADS > 0)
          __builtin_amdgcn_sched_group_barrier(0x008, T::MFMAS - every * T::LOADS, 0);
        if constexpr (T::READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, T::READS, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, T::MFMAS, 0);
      }
      if constexpr (T::JOIN > 0) {
        if (T::JOIN == 1 || (s - s_lo) % T::JOIN == T::JOIN - 1 || s == s_hi - 1)
          static_for<T::WTM>([&](auto i) {
            static_for<T::WTN>([&](auto j) {
              acc[i][j] += part[i][j];
              part[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            });
          });
      }
      buf = buf + 1 == T::STAGES ? 0 : buf + 1;
      if constexpr (T::LAG > 0) buf_a ^= 1; else buf_a = buf;
      // next into the stages of this step
      dma_prep(T::LAG ? buf_a ^ 1 : (buf == 0 ? T::STAGES - 1 : buf - 1),
               buf == 0 ? T::STAGES - 1 : buf - 1);
    }

    int tm, tn;
    tile_at(t, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * T::BM;
    const int64_t n0 = static_cast<int64_t>(tn) * T::BN;
    // Lane holds C[m][n .. n + 3] of each of its tiles: rows r16, columns 4 grp ..
    const int64_t mw = m0 + wm * 16 * T::WTM + r16;
    const int64_t nw = n0 + wn * 16 * T::WTN + 4 * grp;
    const int n_in = static_cast<int>(g.N - nw);   // columns from this lane's first; may be <= 0
    char* scratch = lds + (T::LOOP ? T::RING_BYTES : 0);
    if constexpr (!T::LOOP && (EPI == LE_STATS || (T::STAGED && EPI != LE_PARTIAL))) {
      BDR_WAIT_VM_LGKM(0, 0);   // the trailing zero-filling loads
      BDR_WG_BARRIER();         // and every wave is done with the ring
    }
    // A wave's 16 output rows of one A tile through LDS, then 16 bytes per lane
    // along the rows: whole pieces of OUT_ROW bytes instead of 32-byte ones
    // (1.56 GB written and nothing else: 284 us against 433 us).  The largest
    // tiles have no registers for it and few rows to write per product: directly.
    char* mine = scratch + wave * 16 * T::OUT_PITCH;
    // (d logits: term `term` of the rows)
    const int terms = EPI == LE_DLOGITS ? two : 0;
    auto put_rows = [&](auto ic, int term, auto&& value) {
      if constexpr (!T::STAGED) {
        const int64_t m = mw + decltype(ic)::value * 16;
        static_for<T::WTN>([&](auto j) {
          const int64_t n = nw + decltype(j)::value * 16;
          if (m >= M) return;
          if constexpr (EPI == LE_DLOGITS) {
            if (n < g.ldo)
              store4(static_cast<S*>(g.out) + n / T::KB * g.slab + ((m << terms) + term) * T::KB +
                         n % T::KB,
                     value(j));
          } else if (n < g.N) {
            store4(static_cast<S*>(g.out) + m * g.ldo + n, value(j));
          }
        });
        return;
      }
      static_for<T::WTN>([&](auto j) {
        store4(reinterpret_cast<S*>(mine + r16 * T::OUT_PITCH) + decltype(j)::value * 16 + 4 * grp,
               value(j));
      });
      BDR_WAIT_VM_LGKM(63, 0);
      constexpr bool kOutPanels = EPI == LE_DLOGITS;
      const int64_t left = min<int64_t>(T::BM, M - m0);
      const rsrc_t out =
          kOutPanels
              ? make_rsrc(static_cast<S*>(g.out) + n0 / T::KB * g.slab + (m0 << terms) * T::KB,
                          static_cast<uint32_t>((T::BN / T::KB - 1) * g.slab * ES + (left << terms) * 128))
              : make_rsrc(static_cast<S*>(g.out) + m0 * g.ldo, static_cast<uint32_t>(left * g.ldo * ES));
      const int64_t cols = (kOutPanels ? g.ldo : g.N) - (n0 + wn * 16 * T::WTN);   // may be <= 0
#pragma unroll
      for (int c0 = 0; c0 < 16 * T::OUT_ROW; c0 += 1024) {
        const int c = c0 + lane * 16;
        const int row = c / T::OUT_ROW;
        const int in_row = c % T::OUT_ROW;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(
            mine + (c < 16 * T::OUT_ROW ? row * T::OUT_PITCH + in_row : 0));
        const int m = (wm * T::WTM + decltype(ic)::value) * 16 + row;
        const int nb = wn * T::OUT_ROW + in_row;   // byte of the tile's row
        const uint32_t off =
            kOutPanels ? static_cast<uint32_t>((nb / 128) * g.slab * ES + ((m << terms) + term) * 128 +
                                              nb % 128)
                       : static_cast<uint32_t>((m * g.ldo + n0) * ES + nb);
        const bool ok = c < 16 * T::OUT_ROW && in_row < cols * ES && m < left;
        bstore16(__builtin_bit_cast(f32x4_t, v), out, ok ? off : kOOB);
      }
      BDR_WAIT_VM_LGKM(63, 0);   // read before the next rows are written
    };
    if constexpr (EPI == LE_STATS) {
      // maximum and sum of 2^(x scale2 - maximum) over the tile's columns: lanes,
      // then the four lane groups, then the waves side by side through LDS
      float2* part = reinterpret_cast<float2*>(scratch);   // [WN][BM]
      int lab[T::WTM];   // column of the label, from this lane's first
      static_for<T::WTM>([&](auto i) {
        const int64_t m = mw + decltype(i)::value * 16;
        lab[i] = g.label && m < M ? g.label[m] - g.label0 - static_cast<int>(nw) : -1;
      });
      static_for<T::WTM>([&](auto i) {
        const int64_t m = mw + decltype(i)::value * 16;
        float mx = -INFINITY;
        static_for<T::WTN>([&](auto j) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int n = decltype(j)::value * 16 + c;
            const float z = acc[i][j][c];
            if (n == lab[i]) g.picked[m] = z;
            mx = fmaxf(mx, n < n_in ? z : -INFINITY);
          }
        });
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        mx *= g.scale2;   // positive
        const float ref = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        static_for<T::WTN>([&](auto j) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][c], g.scale2, -ref));
            sum += decltype(j)::value * 16 + c < n_in ? p : 0.f;
          }
        });
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (grp == 0)
          part[wn * T::BM + wm * 16 * T::WTM + decltype(i)::value * 16 + r16] = float2{mx, sum};
      });
      BDR_WAIT_VM_LGKM(63, 0);
      BDR_WG_BARRIER();   // (the next tile's is behind the barrier of its first step)
      for (int r = static_cast<int>(threadIdx.x); r < T::BM; r += 64 * T::WAVES) {
        if (m0 + r >= M) continue;
        float2 v = part[r];
#pragma unroll
        for (int w = 1; w < T::WN; ++w) v = merge_stat(v, part[w * T::BM + r]);
        g.stat[(m0 + r) * g.tiles_n + tn] = v;
      }
    } else if constexpr (EPI == LE_DLOGITS) {
      // rounded to the storage type: the operand of two more matrix products, with as
      // much relative error as their rounded results carry anyway.  That holds for the
      // sum of many roundings; a few rows' may all fall on one side, so a second term
      // takes what the first one's rounding left (16 bits in all), which costs little
      // where the products wait for the weight.  With more rows what is left at the
      // label, by far the largest entry as a rule, is added in fp32 to d hidden and d
      // embedding, and up to kHeldRows rows to the weights' gradients.
      // Columns from N to the padded width hold zeros.
      float l2[T::WTM], cf[T::WTM], corr[T::WTM];
      int lab[T::WTM];   // column of the label, from this lane's first
      static_for<T::WTM>([&](auto i) {   // all before the stores' waits
        const int64_t m = min<int64_t>(mw + decltype(i)::value * 16, M - 1);
        lab[i] = g.label ? g.label[m] - g.label0 - static_cast<int>(nw) : -1;
        l2[i] = g.lse2[m];
        cf[i] = g.coef[m];
        if constexpr (ES == 4) corr[i] = g.lse_corr[m];
      });
      static_for<T::WTM>([&](auto i) {
        auto value = [&](auto j) {
          f32x4_t v;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int n = decltype(j)::value * 16 + c;
            float p = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][c], g.scale2, -l2[i]));
            if constexpr (ES == 4) p *= corr[i];
            v[c] = n < n_in ? cf[i] * (n == lab[i] ? p - 1.f : p) : 0.f;
          }
          return v;
        };
        put_rows(i, 0, [&](auto j) {
          const f32x4_t v = value(j);
          if constexpr (sizeof(S) == 2) {
            const int c = lab[i] - decltype(j)::value * 16;
            const int64_t m = mw + decltype(i)::value * 16;
            if (g.resid && static_cast<unsigned>(c) < 4u && m < M && lab[i] < n_in)
              g.resid[m] = left_over(c == 0 ? v[0] : c == 1 ? v[1] : c == 2 ? v[2] : v[3]);
          }
          return v;
        });
        if constexpr (T::TWO) {
          if (two)
            put_rows(i, 1, [&](auto j) {
              f32x4_t v = value(j);
#pragma unroll
              for (int c = 0; c < 4; ++c) v[c] = left_over(v[c]);
              return v;
            });
        }
      });
    } else if constexpr (EPI == LE_PARTIAL) {
      float* out = static_cast<float*>(g.out) + static_cast<int64_t>(split) * g.slab;
      static_for<T::WTM>([&](auto i) {
        const int64_t m = mw + decltype(i)::value * 16;
        static_for<T::WTN>([&](auto j) {
          const int64_t n = nw + decltype(j)::value * 16;
          if (m < M && n < g.N) {
            f32x4_t* p = reinterpret_cast<f32x4_t*>(out + m * g.ldo + n);
            *p = g.accumulate ? *p + acc[i][j] : acc[i][j];
          }
        });
      });
    } else {
      if constexpr (T::TWO) {
        if (g.resid) {   // rows with their label in this wave's rows of C: resid * operand b
          const int row0 = static_cast<int>(m0) + wm * 16 * T::WTM + g.label0;
          for (int p0 = 0; p0 < live; p0 += 64) {
            int at = -1;
            static_for<kHeld>([&](auto c) { at = p0 == 64 * decltype(c)::value ? held[c] : at; });
            at = at < 0 ? -1 : at - row0;
            unsigned long long hits = __ballot(static_cast<unsigned>(at) < 16u * T::WTM);
            while (hits) {
              const int b = __ffsll(hits) - 1;
              hits &= hits - 1;
              const int rel = __builtin_amdgcn_readlane(at, b);
              const float r = g.resid[p0 + b];
              const S* x = static_cast<const S*>(g.seg[0].b) + static_cast<int64_t>(p0 + b) * g.seg[0].ldb + nw;
              static_for<T::WTM>([&](auto i) {
                if (rel >> 4 == decltype(i)::value && r16 == (rel & 15))
                  static_for<T::WTN>([&](auto j) {
                    if (decltype(j)::value * 16 < n_in)
                      acc[i][j] += r * load4(x + decltype(j)::value * 16);
                  });
              });
            }
          }
        }
      }
      static_for<T::WTM>([&](auto i) { put_rows(i, 0, [&](auto j) { return acc[i][j]; }); });
    }
  }
  BDR_WAIT_VM_LGKM(0, 0);   // the trailing zero-filling loads
}

template <typename T, int EPI>
__global__ __launch_bounds__(64 * T::WAVES, T::SIMD_WAVES) void loss_gemm_kernel(const LossGemm g) {
  loss_gemm_body<T, EPI>(g, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
}

// Two products in one launch, the second one's workgroups after the first's.
template <typename T, int EPI>
__global__ __launch_bounds__(64 * T::WAVES, T::SIMD_WAVES) void loss_gemm_pair_kernel(const LossGemm g0,
                                                                       const LossGemm g1,
                                                                       int blocks0) {
  const int b = static_cast<int>(blockIdx.x);
  const bool second = b >= blocks0;
  loss_gemm_body<T, EPI>(second ? g1 : g0, second ? b - blocks0 : b,
                         second ? static_cast<int>(gridDim.x) - blocks0 : blocks0);
}

// Fills in the tile grid and returns the workgroups of a product.
template <typename T, int EPI>
static int64_t loss_gemm_blocks(LossGemm& g) {
  const int64_t tiles_m = (g.M + T::BM - 1) / T::BM;
  g.tiles_n = static_cast<int>((g.N + T::BN - 1) / T::BN);
  const int64_t items = tiles_m * g.tiles_n * (EPI == LE_PARTIAL ? g.splits : 1);
  const int64_t blocks = (items + 7) / 8 * 8;
  return T::LOOP ? std::min<int64_t>(blocks, 256 * T::PER_CU) : blocks;
}

template <typename T, int EPI>
static hipError_t launch_loss_gemm(LossGemm g, hipStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(loss_gemm_blocks<T, EPI>(g));
  hipLaunchKernelGGL((loss_gemm_kernel<T, EPI>), dim3(blocks), dim3(64 * T::WAVES), 0, stream, g);
  return hipGetLastError();
}

template <typename T, int EPI>
static hipError_t launch_loss_gemm_pair(LossGemm g0, LossGemm g1, hipStream_t stream) {
  const unsigned b0 = static_cast<unsigned>(loss_gemm_blocks<T, EPI>(g0));
  const unsigned b1 = static_cast<unsigned>(loss_gemm_blocks<T, EPI>(g1));
  hipLaunchKernelGGL((loss_gemm_pair_kernel<T, EPI>), dim3(b0 + b1), dim3(64 * T::WAVES), 0, stream,
                     g0, g1, static_cast<int>(b0));
  return hipGetLastError();
}

}  // namespace bdr
