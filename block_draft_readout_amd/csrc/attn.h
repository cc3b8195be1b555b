// Attention of new tokens over a paged cache (gfx950): types, schedule and kernel.
//
//   out[q] = sum_t softmax_t(scale q . k[t]) v[t]  over the positions t that the
//   token sees, in one pass with a running reference r and sum l: a tile of keys
//   gives S = K Q^T, P = 2^(S - r'), and
//   O = O 2^(r - r') + V^T P,  l = l 2^(r - r') + sum P;  out = O / l,
//   where r' is max S if that exceeds r by more than kSlack, else r.
//
// Work.  The query heads that share a kv head read the same keys, so request b's
// n tokens and the `group` heads of a kv head are packed into n * group rows, BM
// of which make a row tile.  A row tile walks its visible keys in tiles of KT.
// Lengths live on the device and differ widely, so the launch has a fixed number
// of workgroups per kv head and each takes an equal, contiguous share of the key
// tiles of all (request, row tile): it finds its place from the lengths by a
// prefix sum.  The workgroups of a share are side by side, one per kv head, and
// read the heads of the same positions at the same time.  A row tile that ends
// up with several workgroups gets partial (O, m, l) in the workspace, which a
// second launch joins in order: nothing depends on the order of arrival.
//
// Products.  S is computed transposed (keys are the rows of the MFMA's result), so
// a lane holds one query's column: its maximum, sum and rescaling are the lane's
// own, and the 32 x 32 result's registers are, rounded to bf16, the operand of the
// second product as they lie (the keys of a step are taken in the order in which
// a lane's registers hold them; V is read with the same order).
// That rounding is half a step of each weight: 2^-8 in bf16, what the output's own
// rounding may be (2^-15 for few rows, whose weights go in as the sum of two bf16), and
// 2^-11 for e4m3 values, which fp16 holds as well as bf16, so that their weights are
// fp16.  The sum l takes the weights before it.  Scores, O, m and l are fp32, and fp32
// tensors have fp32 products throughout (MFMA 32x32x2).
#pragma once

#include <type_traits>

#include "train_device.h"

namespace bdr {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));

struct AttnArgs {
  AttnProblem p;
  int64_t shares;       // of a kv head's work: a workgroup for each and kv head
  int64_t min_share;    // key tiles that a workgroup takes at least
  int whole;            // each row tile is one workgroup's
  float scale2;         // scale * log2(e)
  uint32_t page_magic;  // key / page = mulhi(2 key, page_magic) >> page_shift, keys below 2^30
  int page_shift;
  float* part_o;        // [shares][hkv][2][BM][D]
  float2* part_ml;      // [shares][hkv][2][BM] (m in units of log2, l)
  int32_t* record;      // [shares][hkv][kRecord] what the join needs
};

constexpr int kRecord = 4;   // first row, tokens, row tile, last share (-1: nothing to join)

// -------------------------------------------------------------- schedule
// A request: its rows, row tiles and what they cost in key tiles.  A unit is a row
// tile, or, where causal row tiles differ much, a long and a short one together:
// every unit of a request then costs the same, at most `cost`.
struct AttnSeq {
  int32_t first, n, len;
  int32_t tiles;    // row tiles
  int32_t units;
  int32_t cost;     // key tiles of a unit
  bool paired;
};

template <int BM, int KT>
struct AttnPlan {
  static __device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

  // key tiles [t0, t1) of row tile m (at least one, so that its rows are written)
  static __device__ __forceinline__ void range(const AttnProblem& p, const AttnSeq& s, int m, int& lo,
                                               int& hi, int& t0, int& t1) {
    const int j0 = m * BM / p.group;
    const int j1 = (min((m + 1) * BM, s.n * p.group) - 1) / p.group;
    hi = p.causal ? min(max(s.len - s.n + j1 + 1, 0), s.len) : s.len;
    lo = p.window ? min(max(s.len - s.n + j0 - p.window + 1, 0), hi) : 0;
    t0 = lo / KT;
    t1 = max(div_up(hi, KT), t0 + 1);
  }
  static __device__ __forceinline__ int count(const AttnProblem& p, const AttnSeq& s, int m) {
    int lo, hi, t0, t1;
    range(p, s, m, lo, hi, t0, t1);
    return t1 - t0;
  }

  static __device__ __forceinline__ AttnSeq seq(const AttnProblem& p, int whole, int b) {
    AttnSeq s;
    const int rows = static_cast<int>(p.rows);
    s.first = min(max(p.offsets[b], 0), rows);
    s.n = min(max(p.offsets[b + 1], s.first), rows) - s.first;
    s.len = min(max(p.kv_len[b], 0), p.width * p.page);
    s.tiles = div_up(s.n * p.group, BM);
    s.units = s.tiles;
    s.paired = false;
    if (s.n == 0) {
      s.units = s.cost = 0;
      return s;
    }
    if (whole) {
      s.cost = 1;
      return s;
    }
    const int c0 = count(p, s, 0), c1 = count(p, s, s.tiles - 1);
    if (p.causal && p.window) {
      // a tile of `span` tokens sees at most window + span - 1 positions, in one tile more
      const int span = (BM - 1) / p.group + 2;
      s.cost = static_cast<int>(min(static_cast<int64_t>(max(div_up(s.len, KT), 1)),
                                    (static_cast<int64_t>(p.window) + span) / KT + 2));
    } else {
      s.cost = max(c0, c1);
      // below 7/8 of the longest the shortest row tile is worth pairing
      if (p.causal && s.len >= s.n && s.tiles > 1 && c0 < c1 - c1 / 8) {
        s.paired = true;
        s.units = (s.tiles + 1) / 2;
        const int64_t both = 2 * static_cast<int64_t>(s.len - s.n) +
                             (static_cast<int64_t>(s.tiles + 1) * BM - 2) / p.group + 2;
        s.cost = static_cast<int>(both / KT + 2);
      }
    }
    return s;
  }
  // cost of the whole request
  static __device__ __forceinline__ int64_t total(const AttnSeq& s) {
    return static_cast<int64_t>(s.units) * s.cost;
  }
};

__device__ __forceinline__ int64_t wave_sum_i64(int64_t v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ int64_t uniform_i64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// -------------------------------------------------------------- kernel
// Many rows: WM waves hold 32 rows each and share the tiles of keys in LDS.
template <typename C_, typename S_, int D_, int WM_, int KT_>
struct AttnMany {
  using C = C_;                       // cache element: uint16_t (bf16), uint8_t (e4m3) or float
  using S = S_;                       // queries, output and LDS: uint16_t or float
  static constexpr bool kFew = false, kTall = false;
  static constexpr int D = D_, WM = WM_, RT = 1;
  static constexpr int KT = KT_;      // keys of a tile (D 256: 64 would be 453 us where 32 are 398)
  static constexpr int THREADS = 64 * WM;
  static constexpr int BM = 32 * WM * RT;
  static constexpr int CS = static_cast<int>(sizeof(C)), ES = static_cast<int>(sizeof(S));
  static constexpr int ROWB = D * ES;                    // bytes of an LDS row
  static constexpr int PER16 = 16 / CS;                  // cache elements of 16 bytes
  static constexpr int CPR = D / PER16;                  // 16-byte pieces of a cache row
  static constexpr int LOADS = KT * CPR / THREADS;       // 16-byte loads of a thread, K or V
  static constexpr int RPL = CPR > 64 ? 1 : 64 / CPR;    // rows of a wave's load
  static constexpr int TILE_BYTES = KT * ROWB;           // K or V of a tile
  static constexpr int LDS_BYTES = 4 * TILE_BYTES;       // two buffers
  static constexpr int QN = ROWB / 32;                   // 16-byte query pieces of a lane and row
  static constexpr int SIMD_WAVES = RT == 1 && LDS_BYTES <= 80 * 1024 && D * ES <= 256 ? 2 : 1;
  static_assert(KT % 32 == 0 && KT <= 64, "a lane looks up one key's page");
  static_assert(LOADS * THREADS == KT * CPR, "loads split evenly");
  static_assert(LDS_BYTES <= 160 * 1024, "tile fits");
};

// Very many rows: eight waves, two of a SIMD in opposite phases (see the body).
template <typename C_, typename S_, int D_, int KT_>
struct AttnTall : AttnMany<C_, S_, D_, 8, KT_> {
  using Base = AttnMany<C_, S_, D_, 8, KT_>;
  static constexpr bool kTall = true;
  static constexpr int LDS_BYTES = 7 * Base::TILE_BYTES;   // three buffers of keys, four of values
  static constexpr int SIMD_WAVES = 2;
};

// Few rows: WN waves hold the same RT x 16 rows and walk key tiles of their own, each through
// LDS of its own, joined at the end.  Tiles come straight from the cache to LDS as they are
// stored there.
template <typename C_, typename S_, int D_, int RT_, int WN_>
struct AttnFew {
  using C = C_;
  using S = S_;
  static constexpr bool kFew = true, kTall = false;
  static constexpr int D = D_, RT = RT_;
  static constexpr int CS = static_cast<int>(sizeof(C)), ES = static_cast<int>(sizeof(S));
  static constexpr int ROWB = D * CS;                    // bytes of an LDS row
  static constexpr int KT = CS == 1 ? 64 : 32;
  static constexpr int WN = WN_;
  static constexpr int THREADS = 64 * WN;
  static constexpr int BM = 16 * RT;
  static constexpr int CPR = ROWB / 16;                  // 16-byte chunks of a row
  static constexpr int RPL = 64 / CPR;                   // rows of a wave's load
  static constexpr int LOADS = KT / RPL;
  static constexpr int TILE_BYTES = KT * ROWB;
  // Two waves of a SIMD cover each other's waits; where registers are for one, it has two tiles in
  // LDS, and the next one's loads are in flight under a whole tile's work.
  static constexpr bool kTwo = D * RT <= (CS == 1 ? 256 : 384);
  static constexpr int BUFS = D == 128 && !kTwo && WN_ == 4 ? 2 : 1;
  static constexpr int WAVE_BYTES = 2 * TILE_BYTES * BUFS;   // (a wave's O of 16 rows, fp32, fits)
  // Queries stay in LDS where two waves of a SIMD have no registers for them.
  static constexpr bool QLDS = D == 128 && RT >= 3;
  static constexpr int Q_AT = WAVE_BYTES * WN;
  static constexpr int PAGE_AT = Q_AT + (QLDS ? BM * D * ES : 0);   // page ids of a tile, 256 bytes a wave
  static constexpr int LDS_BYTES = PAGE_AT + 256 * WN;
  static constexpr int QN = D * ES / 64;                 // 16-byte query pieces of a lane and row
  // bf16 terms of a weight.  The second one's products fit under the cache's loads (16 x 8 rows
  // over up to 32768 positions 179.7 against 182.0 us, one token over 1000 12.7 against 13.3), but
  // not where four tiles of 128 have a SIMD's registers for one wave (104 against 118 us), nor
  // under many rows (2048 tokens over 16384: 515 against 758 us; D 256: 395 against 478).
  static constexpr int TERMS = CS == 2 && (D * RT <= 384 || D == 256) ? 2 : 1;
  static constexpr int SIMD_WAVES = WN == 8 || (LDS_BYTES <= 80 * 1024 && kTwo) ? 2 : 1;
  static_assert(CPR <= 64 && KT % RPL == 0, "a load is whole rows");
  static_assert(16 * D * 4 + 128 <= WAVE_BYTES, "a wave's output and statistics fit its tiles' place");
  static_assert(LDS_BYTES <= 160 * 1024, "tiles fit");
  static_assert(2 * LOADS + 1 < 64, "loads in flight can be counted");
};

// Places of the 16-byte chunks c of LDS row r: an XOR by the row, so that the lanes of one
// pass meet distinct banks.  Keys: 16 lanes read one chunk of 16 rows.
template <int ROWB>
__device__ __forceinline__ uint32_t key_turn(uint32_t r) {
  return ROWB >= 256 ? r & 15u : ROWB == 128 ? (r >> 1) & 7u : (r >> 2) & 3u;
}
template <int ROWB>
__device__ __forceinline__ uint32_t key_place(uint32_t r, uint32_t c) {
  return r * ROWB + ((c ^ key_turn<ROWB>(r)) << 4);
}
// Values: what a pass of 32 lanes reads depends on the kind of read.
template <typename T>
__device__ __forceinline__ uint32_t value_turn(uint32_t r) {
  constexpr int ROWB = T::ROWB;
  if constexpr (!T::kFew)                           // 64 bytes of rows r .. r + 3
    return ROWB >= 256 ? (r & 3u) << 2 : (r & 2u) << 1;
  else if constexpr (sizeof(typename T::C) == 2)    // 32 bytes of rows r .. r + 7
    return ROWB >= 256 ? (r & 7u) << 1 : r & 6u;
  else if constexpr (sizeof(typename T::C) == 4)    // 64 bytes of rows r, r + 4, r + 8, r + 12
    return ((r >> 2) & 3u) << 2;
  else                                              // 16 bytes of rows r .. r + 7 and r + 16 .. r + 23
    return ROWB >= 256 ? (r & 7u) | ((r >> 1) & 8u)
                       : ROWB == 128 ? ((r >> 1) & 3u) | ((r >> 2) & 4u) : ((r >> 2) & 1u) | ((r >> 3) & 2u);
}
template <typename T>
__device__ __forceinline__ uint32_t value_place(uint32_t r, uint32_t c) {
  return r * T::ROWB + ((c ^ value_turn<T>(r)) << 4);
}

// 8 e4m3 codes as bf16 (every code's value is one)
__device__ __forceinline__ bf16x8_t widen8(uint32_t v, uint32_t w) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// and 16
__device__ __forceinline__ void widen16(u32x4_t v, u32x4_t& a, u32x4_t& b) {
  a = __builtin_bit_cast(u32x4_t, widen8(v.x, v.y));
  b = __builtin_bit_cast(u32x4_t, widen8(v.z, v.w));
}

// Values and their weights as the second product takes them: bf16, or fp16 where the cache holds
// e4m3 codes (every code's value is one, and a weight keeps 11 bits for 8 at the same rate).
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
__device__ __forceinline__ bf16x8_t widen8_half(uint32_t v, uint32_t w) {   // 16 bits each, whatever their type
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, false);
  const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, true);
  const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
  const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
  return __builtin_bit_cast(bf16x8_t, f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]});
}
template <typename C>
__device__ __forceinline__ uint32_t pack_weights(float x, float y) {
  if constexpr (sizeof(C) == 1) {
    typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, f16x2_t{static_cast<_Float16>(x), static_cast<_Float16>(y)});
  } else {
    return pack_bf16(x, y);
  }
}
// Two terms of bf16 weights: their upper bits and the rest, at most 2^-7 of them and rounded.  Neither
// is negative, and the rest, a last bit of fp32 too large, is 0 with the weight alone: an infinite
// value stays infinite.
__device__ __forceinline__ uint2 split_weights(float x, float y) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  return uint2{__builtin_amdgcn_perm(b, a, 0x07060302u),
               pack_bf16(fmaf(x, 1.f + 0x1p-23f, -__uint_as_float(a & 0xFFFF0000u)),
                         fmaf(y, 1.f + 0x1p-23f, -__uint_as_float(b & 0xFFFF0000u)))};
}
template <typename C>
__device__ __forceinline__ f32x4_t weigh(bf16x8_t v, u32x4_t w, f32x4_t o) {
  if constexpr (sizeof(C) == 1)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, v), __builtin_bit_cast(f16x8_t, w), o, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8_t, w), o, 0, 0, 0);
}
template <typename C>
__device__ __forceinline__ f32x16_t weigh(bf16x8_t v, u32x4_t w, f32x16_t o) {
  if constexpr (sizeof(C) == 1)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, v), __builtin_bit_cast(f16x8_t, w), o, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf16x8_t, w), o, 0, 0, 0);
}

// A lane's key of a tile to come.  The page's id is asked for behind the loads of an earlier
// tile and used after those have been waited for: an address that depends on it never holds up a
// tile.
struct AttnPage {
  int32_t id;
  int32_t place;   // in the page; -1: the key is not read
};

// The reference that a row's exponentials are taken against follows the row's maximum only where
// that has grown by more than kSlack (a factor of 2^8): probabilities are 256 at most then, which
// costs no precision in floating point, and sums of 2^31 of them stay in range.  The maximum of
// random scores still grows in every second of the first hundred tiles, and a new reference scales
// all sums.  Nothing seen yet: a reference of 0.
// fp16 weights are taken 2^7 larger (2^15 at most): those down to 2^-21 of the reference's keep all
// their bits.  Sums and partials hold that factor too; it cancels in out, and lse takes it out.
constexpr float kSlack = 8.f;
template <typename C>
constexpr float kLift = sizeof(C) == 1 ? 7.f : 0.f;
template <typename C>
constexpr float kDown = sizeof(C) == 1 ? 0x1p-7f : 1.f;
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }

// What the queries take over from the scores' factor, so that it is a positive number, as the
// running maximum wants it: the sign, or that it is no number (the scale of a head's keys).  Keys
// that a row does not see stay out of it that way.
struct AttnSign {
  bool flip, nan;
};
template <typename C>
__device__ __forceinline__ AttnSign positive(float& scale2) {
  const bool nan = sizeof(C) == 1 && !(fabsf(scale2) < INFINITY);   // (the call's own scale is a number)
  const bool flip = scale2 < 0.f;
  scale2 = nan ? 1.f : fmaxf(fabsf(scale2), 0x1p-126f);   // (0 times a masked score is no number)
  return AttnSign{flip, nan};
}

// What both kinds of kernels share.
template <typename T>
struct AttnLoader {
  using S = typename T::S;
  using C = typename T::C;

  // column of the table and place in the page
  static __device__ __forceinline__ uint32_t column_of(const AttnArgs& g, int key0, int lo, int hi, int lane,
                                                       int32_t& place) {
    const int key = key0 + (T::KT == 64 ? lane : lane & 31);
    const int at = max(min(max(key, lo), hi - 1), 0);   // (a key of the table, whatever lo and hi)
    const uint32_t col = __umulhi(2u * at, g.page_magic) >> g.page_shift;
    place = key == at && key < hi ? static_cast<int32_t>(at - col * g.p.page) : -1;
    return col;
  }
  static __device__ __forceinline__ AttnPage page_of(const AttnArgs& g, const int32_t* table, int key0, int lo,
                                                     int hi, int lane) {
    AttnPage a;
    a.id = table[column_of(g, key0, lo, hi, lane, a.place)];
    return a;
  }
  // its bytes from the head's first, 0 and false where it is not read
  static __device__ __forceinline__ uint64_t offset_of(const AttnProblem& p, AttnPage a, bool& in) {
    in = a.place >= 0 && static_cast<uint32_t>(a.id) < static_cast<uint32_t>(p.pages);
    const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(a.id)) * p.page_bytes +
                         static_cast<uint64_t>(static_cast<uint32_t>(a.place)) * p.token_bytes;
    return in ? off : 0;
  }
  // rows of one load lie in one page, its offsets in 32 bits
  static __device__ __forceinline__ bool whole_loads(const AttnProblem& p) {
    return p.page % T::RPL == 0 && p.token_bytes < (1u << 31) / 64;
  }

  // A lane's 16-byte pieces of row r of the packed rows: features place(i) on.
  template <int QN, typename Place>
  static __device__ __forceinline__ void load_q(const AttnProblem& p, const AttnSeq& s, int h, int r, Place place,
                                                AttnSign f, u32x4_t (&q)[QN]) {
    const bool in = r < s.n * p.group;
    const int j = in ? r / p.group : 0;
    const int head = in ? h * p.group + (r - j * p.group) : 0;
    const S* at = static_cast<const S*>(p.q) + static_cast<int64_t>(s.first + j) * p.q_row +
                  static_cast<int64_t>(head) * p.q_head;
    // (of all types: queries that nothing touches here would be waited for in the loop over the keys, and each
    // tile's loads with them: 426 us for 396, 24 requests' chunks over 12000 bf16 keys of 256)
    const uint32_t sign = f.flip ? (T::ES == 2 ? 0x80008000u : 0x80000000u) : 0u;
    const uint32_t nan = f.nan ? (T::ES == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu) : 0u;
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const u32x4_t v = in ? load16(at + place(i)) : u32x4_t{0, 0, 0, 0};
      q[i] = u32x4_t{(v.x ^ sign) | nan, (v.y ^ sign) | nan, (v.z ^ sign) | nan, (v.w ^ sign) | nan};
    }
  }

  // four features of an output row: out = o / l
  static __device__ __forceinline__ void put(const AttnArgs& g, int first, int h, int r, int d, f32x4_t o,
                                             float m, float l, float v_scale) {
    const AttnProblem& p = g.p;
    const int j = r / p.group;
    const int head = h * p.group + (r - j * p.group);
    const int64_t row = (static_cast<int64_t>(first) + j) * p.hq + head;
    const float inv = l == 0.f ? 0.f : v_scale / l;   // (NaN stays)
    S* out = static_cast<S*>(p.out) + row * T::D + d;
    if constexpr (T::ES == 2)
      *reinterpret_cast<uint2*>(out) = uint2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
    else
      *reinterpret_cast<f32x4_t*>(out) = f32x4_t{o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
    if (p.lse && d == 0)
      p.lse[row] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l * kDown<C>)) * kLn2;
  }
};

// Scores of a lane's column: mask, running maximum and sum, probabilities in place.  N values of
// keys key0 + key_of(i); `fold` takes the maximum over the lanes that hold the column's other keys.
// Returns the factor of what was summed before.
template <typename C, int N, typename KeyOf, typename Fold>
__device__ __forceinline__ float softmax_step(float (&s)[N], bool edge, int lo, int hi, float scale2, KeyOf key_of,
                                              Fold fold, float& m, float& l) {
  if (edge) {
    asm volatile("");   // (a branch: few tiles lie on an edge)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int key = key_of(i);
      if (key < lo || key >= hi) s[i] = -INFINITY;
    }
  }
  float top = s[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, s[i]);
  const float most = fold(top) * scale2;
  const float next = most > m + kSlack ? most : m;
  const float ref = reference(next);
  const float f = __builtin_amdgcn_exp2f(m - ref);
  m = next;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], scale2, kLift<C> - ref));
    sum += s[i];
  }
  l = l * f + sum;
  return f;
}

// maximum over lanes l, l ^ 32 (and l ^ 16)
__device__ __forceinline__ float max_xor32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_xor16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// four 16-bit values of column lane % 16 from 4 rows x 16 columns that a group of 16 lanes names,
// 8 bytes each
__device__ __forceinline__ i16x4_t read_tr(const char* p) {
  typedef __attribute__((address_space(3))) i16x4_t* lds_t;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)p);
}
__device__ __forceinline__ bf16x8_t join_tr(i16x4_t x, i16x4_t y) {
  typedef short i16x8_t __attribute__((ext_vector_type(8)));
  const i16x8_t a = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8_t, a);
}

// -------------------------------------------------------------- many rows
// Tiles go cache -> registers -> LDS, in two buffers, with one barrier a tile; the two waves of a
// SIMD run the matrix unit and the vector unit (exponentials) in turn.
template <typename T>
struct AttnManyBody : AttnLoader<T> {
  using L = AttnLoader<T>;
  using S = typename T::S;
  using C = typename T::C;

  // What a thread holds of a tile of keys and values.
  struct Stage {
    u32x4_t k[T::LOADS], v[T::LOADS];
    uint64_t live;                  // bit t: row t of the tile is read (others are zeros)
  };
  static constexpr uint64_t kAll = T::KT == 64 ? ~0ull : 0xFFFFFFFFull;

  // Every lane looks a key up; a load's rows take their offsets from the lanes that did.  Where
  // they lie in one page, one offset is the load's own scalar.
  // off, live: what offset_of gave the lanes
  static __device__ __forceinline__ void load_at(const AttnProblem& p, const char* kb, const char* vb, uint64_t off,
                                                 uint64_t live, int tid, Stage& g) {
    // a row that is not read takes the first page's first row, and is cleared on its way to LDS
    const int lo = static_cast<int>(off), hi = static_cast<int>(off >> 32);
    asm volatile("" : "+v"(tid));   // (offsets are made anew rather than held over the loop)
    const uint32_t c = static_cast<uint32_t>(tid % T::CPR) * 16;
    g.live = live;
    if (live == kAll && L::whole_loads(p)) {
      const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
      const uint32_t mine = (tid & 63) / T::CPR * p.token_bytes + c;
#pragma unroll
      for (int i = 0; i < T::LOADS; ++i) {
        const int row = (64 * wave + T::THREADS * i) / T::CPR;
        const uint32_t l = __builtin_amdgcn_readlane(lo, row), h = __builtin_amdgcn_readlane(hi, row);
        const uint64_t at = (static_cast<uint64_t>(h) << 32) | l;
        g.k[i] = load16(kb + at + mine);
        g.v[i] = load16(vb + at + mine);
      }
    } else {
#pragma unroll
      for (int i = 0; i < T::LOADS; ++i) {
        const int row = (tid + T::THREADS * i) / T::CPR;
        const uint32_t l = __shfl(lo, row), h = __shfl(hi, row);
        const uint64_t at = (static_cast<uint64_t>(h) << 32) | l;
        g.k[i] = load16(kb + at + c);
        g.v[i] = load16(vb + at + c);
      }
    }
  }
  static __device__ __forceinline__ void load(const AttnProblem& p, const char* kb, const char* vb, AttnPage a,
                                              int tid, Stage& g) {
    bool in;
    const uint64_t off = L::offset_of(p, a, in);
    load_at(p, kb, vb, off, __ballot(in) & kAll, tid, g);
  }

  template <typename Keys>
  static __device__ __forceinline__ void store16(char* lds, uint32_t at, uint32_t at_next, u32x4_t v, Keys) {
    if constexpr (T::CS == 1) {
      u32x4_t x, y;
      if constexpr (Keys::value) {
        widen16(v, x, y);
      } else {
        x = __builtin_bit_cast(u32x4_t, widen8_half(v.x, v.y));
        y = __builtin_bit_cast(u32x4_t, widen8_half(v.z, v.w));
      }
      *reinterpret_cast<u32x4_t*>(lds + at) = x;
      *reinterpret_cast<u32x4_t*>(lds + at_next) = y;
    } else {
      *reinterpret_cast<u32x4_t*>(lds + at) = v;
    }
  }
  // rows that are not read become zeros
  static __device__ __forceinline__ void clear(int tid, Stage& g) {
    asm volatile("");   // (a branch: rare)
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i)
      if (!((g.live >> ((tid + T::THREADS * i) / T::CPR)) & 1)) g.k[i] = g.v[i] = u32x4_t{0, 0, 0, 0};
  }
  template <typename Keys>   // true_type: keys' places, false_type: values'
  static __device__ __forceinline__ void store_one(char* lds, int tid, const u32x4_t (&x)[T::LOADS], Keys) {
    constexpr int W = T::ES / T::CS;   // 16-byte chunks in LDS of a piece
    auto place = [](uint32_t r, uint32_t c) {
      if constexpr (Keys::value) return key_place<T::ROWB>(r, c);
      else return value_place<T>(r, c);
    };
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
      const int idx = tid + T::THREADS * i;
      const uint32_t row = idx / T::CPR, c = W * (idx % T::CPR);
      store16(lds, place(row, c), place(row, c + W - 1), x[i], Keys{});
    }
  }
  static __device__ __forceinline__ void store(char* lk, char* lv, int tid, Stage& g) {
    if (g.live != kAll) clear(tid, g);
    store_one(lk, tid, g.k, std::true_type{});
    store_one(lv, tid, g.v, std::false_type{});
  }

  // 16-byte operand pieces of 32 keys: piece i is chunk 2 i + lane / 32 of key lane % 32
  static __device__ __forceinline__ void read_keys(const char* lk, int sub, int lane, u32x4_t (&k)[T::QN]) {
    const uint32_t row = 32 * sub + (lane & 31);
#pragma unroll
    for (int i = 0; i < T::QN; ++i) k[i] = load16(lk + key_place<T::ROWB>(row, 2 * i + (lane >> 5)));
  }

  // S^T of 32 keys against the wave's queries: keys 8 (r / 4) + 4 (lane / 32) + r % 4 of query lane % 32
  static __device__ __forceinline__ void scores(const u32x4_t (&k)[T::QN], const u32x4_t (&q)[T::RT][T::QN],
                                                f32x16_t (&c)[T::RT]) {
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) c[rt] = f32x16_t{};
#pragma unroll
    for (int i = 0; i < T::QN; ++i) {
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt) {
        if constexpr (T::ES == 2) {
          c[rt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8_t, k[i]), __builtin_bit_cast(bf16x8_t, q[rt][i]), c[rt], 0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            c[rt] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(k[i][e]), __uint_as_float(q[rt][i][e]),
                                                         c[rt], 0, 0, 0);
        }
      }
    }
  }

  // Operand pieces of 16 values (16 bits each): features 32 i + lane % 32 of the keys that a lane's
  // probabilities are of
  static __device__ __forceinline__ void read_values(const char* lv, int sub, int ks, int lane,
                                                     bf16x8_t (&v)[T::D / 32]) {
    const uint32_t row = 32 * sub + 16 * ks + 4 * (lane >> 5) + ((lane & 15) >> 2);
#pragma unroll
    for (int i = 0; i < T::D / 32; ++i) {
      const uint32_t c = 4 * i + ((lane >> 3) & 2) + ((lane >> 1) & 1);
      v[i] = join_tr(read_tr(lv + value_place<T>(row, c) + (lane & 1) * 8),
                     read_tr(lv + value_place<T>(row + 8, c) + (lane & 1) * 8));
    }
  }

  // O^T += V^T P^T of 16 keys: registers 8 ks .. 8 ks + 7 of the probabilities
  static __device__ __forceinline__ void add_values(const bf16x8_t (&v)[T::D / 32], int ks,
                                                    const f32x16_t (&p)[T::RT], f32x16_t (&o)[T::RT][T::D / 32]) {
    u32x4_t b[T::RT];
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt)
#pragma unroll
      for (int e = 0; e < 4; ++e) b[rt][e] = pack_weights<C>(p[rt][8 * ks + 2 * e], p[rt][8 * ks + 2 * e + 1]);
#pragma unroll
    for (int i = 0; i < T::D / 32; ++i)
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt)
        o[rt][i] = weigh<C>(v[i], b[rt], o[rt][i]);
  }
  // (fp32: straight from LDS)
  static __device__ __forceinline__ void add_values_f32(const char* lv, int sub, int lane, const f32x16_t (&p)[T::RT],
                                                        f32x16_t (&o)[T::RT][T::D / 32]) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const uint32_t row = 32 * sub + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
#pragma unroll
      for (int i = 0; i < T::D / 32; ++i) {
        const uint32_t d = 32 * i + (lane & 31);
        const float a = *reinterpret_cast<const float*>(lv + value_place<T>(row, d / 4) + (d & 3) * 4);
#pragma unroll
        for (int rt = 0; rt < T::RT; ++rt)
          o[rt][i] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, p[rt][r], o[rt][i], 0, 0, 0);
      }
    }
  }

  // a wave's rows, from row `first` of the tile on: the output, or a partial in `slot`
  static __device__ __forceinline__ void put_rows(const AttnArgs& g, const AttnSeq& s, int h, int m, int first,
                                                  int lane, int64_t slot, const f32x16_t (&o)[T::RT][T::D / 32],
                                                  const float (&mx)[T::RT], const float (&l)[T::RT], float v_scale) {
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) {
      const int rl = first + 32 * rt + (lane & 31);   // row in the tile
      const int r = m * T::BM + rl;
      if (r < s.n * g.p.group) {
        if (slot >= 0 && lane < 32) g.part_ml[slot * T::BM + rl] = float2{mx[rt], l[rt]};
#pragma unroll
        for (int i = 0; i < T::D / 32; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int d = 32 * i + 8 * x + 4 * (lane >> 5);
            const f32x4_t v = {o[rt][i][4 * x], o[rt][i][4 * x + 1], o[rt][i][4 * x + 2], o[rt][i][4 * x + 3]};
            if (slot >= 0)
              *reinterpret_cast<f32x4_t*>(g.part_o + (slot * T::BM + rl) * T::D + d) = v;
            else
              L::put(g, s.first, h, r, d, v, mx[rt], l[rt], v_scale);
          }
      }
    }
  }

  // One row tile over key tiles [ta, tb).  slot < 0: the output itself, else a partial there.
  static __device__ __forceinline__ void run(const AttnArgs& g, const AttnSeq& s, int b, int h, int m, int ta,
                                             int tb, int lo, int hi, int64_t slot, char* lds) {
    const AttnProblem& p = g.p;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int tid = static_cast<int>(threadIdx.x);
    const int r0 = m * T::BM + wave * 32 * T::RT;
    const int rows = s.n * p.group;
    float scale2 = g.scale2, v_scale = 1.f;
    if constexpr (sizeof(C) == 1) {
      scale2 *= p.k_scale[h];
      v_scale = p.v_scale[h];
    }
    const AttnSign sign = positive<C>(scale2);

    const int32_t* table = p.table + static_cast<int64_t>(b) * p.width;
    const char* kb = static_cast<const char*>(p.k_cache) + h * p.head_bytes;
    const char* vb = static_cast<const char*>(p.v_cache) + h * p.head_bytes;
    char* now = lds;                             // keys and values of a tile
    char* other = lds + 2 * T::TILE_BYTES;
    Stage stage;
    AttnPage page = L::page_of(g, table, ta * T::KT, lo, hi, lane);
    load(p, kb, vb, page, tid, stage);
    page = L::page_of(g, table, (ta + 1) * T::KT, lo, hi, lane);

    u32x4_t q[T::RT][T::QN];
    int row_lo[T::RT], row_hi[T::RT];
    f32x16_t o[T::RT][T::D / 32];
    float mx[T::RT], l[T::RT];
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) {
      const int r = r0 + 32 * rt + (lane & 31);
      L::load_q(p, s, h, r, [&](int i) { return (2 * i + (lane >> 5)) * (16 / T::ES); }, sign, q[rt]);
      const int at = s.len - s.n + r / p.group;
      row_hi[rt] = p.causal ? min(at + 1, s.len) : s.len;
      row_lo[rt] = p.window ? at - p.window + 1 : 0;
      mx[rt] = -INFINITY;
      l[rt] = 0.f;
#pragma unroll
      for (int i = 0; i < T::D / 32; ++i) o[rt][i] = f32x16_t{};
    }
    // the wave's rows all see the keys [see_lo, see_hi)
    const int first = s.len - s.n + r0 / p.group;
    const int last = s.len - s.n + min(r0 + 32 * T::RT - 1, rows - 1) / p.group;
    const int see_hi = p.causal ? min(first + 1, s.len) : s.len;
    const int see_lo = p.window ? last - p.window + 1 : 0;

    constexpr int SUB = T::KT / 32;
    // Where a wave has all registers of its SIMD the sums stay in accumulation registers, which only
    // a new reference reads; left alone they are moved there and back with every tile (458 us
    // against 412: 24 requests' chunks over 12000 bf16 keys of 256, a window of 4096).
    auto hold = [&]() {
      if constexpr (T::D == 256) {
#pragma unroll
        for (int rt = 0; rt < T::RT; ++rt)
#pragma unroll
          for (int i = 0; i < T::D / 32; ++i) asm volatile("" : "+a"(o[rt][i]));
      }
    };
    for (int t = ta; t < tb; ++t) {
      hold();
      store(now, now + T::TILE_BYTES, tid, stage);
      if (t + 1 < tb) {
        load(p, kb, vb, page, tid, stage);
        page = L::page_of(g, table, (t + 2) * T::KT, lo, hi, lane);
      }
      // one barrier a tile: the buffer written next was last read before the barrier after that
      __syncthreads();
      const char* lk = now;
      const char* lv = now + T::TILE_BYTES;
      now = other;
      other = const_cast<char*>(lk);
      if (r0 >= rows) continue;
      const int key0 = t * T::KT;
      f32x16_t sc[SUB][T::RT];
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        u32x4_t k[T::QN];
        read_keys(lk, u, lane, k);
        scores(k, q, sc[u]);
      }
      // operands of the next 32 keys are asked for while these are multiplied
      __builtin_amdgcn_sched_group_barrier(0x100, T::QN, 0);
#pragma unroll
      for (int i = 0; i < T::QN * (SUB - 1); ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, T::RT, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x8, T::RT * T::QN, 0);
      if (key0 < see_lo || key0 + T::KT > see_hi) {
        asm volatile("");   // (a branch: few tiles lie on an edge)
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int key = key0 + 32 * u + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
#pragma unroll
            for (int rt = 0; rt < T::RT; ++rt)
              if (key < row_lo[rt] || key >= row_hi[rt]) sc[u][rt][r] = -INFINITY;
          }
      }
      float most[T::RT], ref[T::RT];
      bool grew = false;
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt) {
        float top = sc[0][rt][0];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[u][rt][r]);
        most[rt] = fmaxf(mx[rt], max_xor32(top) * scale2);
        grew = grew || most[rt] > mx[rt] + kSlack;
      }
      hold();
      if (__any(grew)) {
        asm volatile("");
#pragma unroll
        for (int rt = 0; rt < T::RT; ++rt) {
          const float f = __builtin_amdgcn_exp2f(mx[rt] - reference(most[rt]));
          mx[rt] = most[rt];
          l[rt] *= f;
#pragma unroll
          for (int i = 0; i < T::D / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[rt][i][r] *= f;
        }
        hold();
      }
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt) ref[rt] = reference(mx[rt]) - kLift<C>;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
#pragma unroll
        for (int rt = 0; rt < T::RT; ++rt) {
          float sum = 0.f;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            sc[u][rt][r] = __builtin_amdgcn_exp2f(fmaf(sc[u][rt][r], scale2, -ref[rt]));
            sum += sc[u][rt][r];
          }
          l[rt] += sum;
        }
        if constexpr (T::ES == 2) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            bf16x8_t v[T::D / 32];
            read_values(lv, u, ks, lane, v);
            add_values(v, ks, sc[u], o);
          }
        } else {
          add_values_f32(lv, u, lane, sc[u], o);
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) l[rt] += __shfl_xor(l[rt], 32);
    put_rows(g, s, h, m, wave * T::RT * 32, lane, slot, o, mx, l, v_scale);
    __syncthreads();   // the tiles in LDS are read: the next row tile may overwrite them
  }
};

// -------------------------------------------------------------- very many rows
// Waves w and w + 4 share a SIMD.  A wave goes through two phases a tile: softmax (with the
// copies: a tile's way through registers to LDS) and products (this tile's values, the next one's
// scores).  The second four waves start one barrier late, so at any time one wave of a SIMD has
// the matrix unit and the other the vector unit; a barrier ends every phase.
template <typename T>
struct AttnTallBody : AttnManyBody<T> {
  using M = AttnManyBody<T>;
  using L = AttnLoader<T>;
  using S = typename T::S;
  using C = typename T::C;
  static constexpr int SUB = T::KT / 32;

  static __device__ __forceinline__ void run(const AttnArgs& g, const AttnSeq& s, int b, int h, int m, int ta,
                                             int tb, int lo, int hi, int64_t slot, char* lds) {
    const AttnProblem& p = g.p;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int tid = static_cast<int>(threadIdx.x);
    const int r0 = m * T::BM + wave * 32;
    const int rows = s.n * p.group;
    float scale2 = g.scale2, v_scale = 1.f;
    if constexpr (sizeof(C) == 1) {
      scale2 *= p.k_scale[h];
      v_scale = p.v_scale[h];
    }
    const AttnSign sign = positive<C>(scale2);

    const int32_t* table = p.table + static_cast<int64_t>(b) * p.width;
    const char* kb = static_cast<const char*>(p.k_cache) + h * p.head_bytes;
    const char* vb = static_cast<const char*>(p.v_cache) + h * p.head_bytes;
    // buffers of keys: of the next tile, the one after, and to fill; of values: of this tile, the
    // next two, and to fill
    char* k1 = lds + T::TILE_BYTES;
    char* k2 = lds + 2 * T::TILE_BYTES;
    char* k3 = lds;
    char* v0 = lds + 3 * T::TILE_BYTES;
    char* v1 = lds + 4 * T::TILE_BYTES;
    char* v2 = lds + 5 * T::TILE_BYTES;
    char* v3 = lds + 6 * T::TILE_BYTES;

    typename M::Stage stage;
    {
      typename M::Stage x0;
      const AttnPage p0 = L::page_of(g, table, ta * T::KT, lo, hi, lane);
      const AttnPage p1 = L::page_of(g, table, (ta + 1) * T::KT, lo, hi, lane);
      M::load(p, kb, vb, p0, tid, x0);
      M::load(p, kb, vb, p1, tid, stage);
      M::store(k3, v0, tid, x0);
      M::store(k1, v1, tid, stage);
    }
    AttnPage page = L::page_of(g, table, (ta + 2) * T::KT, lo, hi, lane);
    M::load(p, kb, vb, page, tid, stage);   // of tile t + 2 from here on
    page = L::page_of(g, table, (ta + 3) * T::KT, lo, hi, lane);

    u32x4_t q[1][T::QN];
    L::load_q(p, s, h, r0 + (lane & 31), [&](int i) { return (2 * i + (lane >> 5)) * (16 / T::ES); }, sign, q[0]);
    const int at = s.len - s.n + (r0 + (lane & 31)) / p.group;
    const int row_hi = p.causal ? min(at + 1, s.len) : s.len;
    const int row_lo = p.window ? at - p.window + 1 : 0;
    f32x16_t o[1][T::D / 32];
    float mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < T::D / 32; ++i) o[0][i] = f32x16_t{};
    // the wave's rows all see the keys [see_lo, see_hi)
    const int first = s.len - s.n + r0 / p.group;
    const int last = s.len - s.n + min(r0 + 31, rows - 1) / p.group;
    const int see_hi = p.causal ? min(first + 1, s.len) : s.len;
    const int see_lo = p.window ? last - p.window + 1 : 0;

    __syncthreads();
    if (wave >= 4) __syncthreads();

    f32x16_t sc[SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      u32x4_t k[T::QN];
      M::read_keys(k3, u, lane, k);
      f32x16_t c[1];
      M::scores(k, q, c);
      sc[u] = c[0];
    }
    for (int t = ta; t < tb; ++t) {
      // ---- softmax
      u32x4_t pr[SUB][2];   // probabilities, as the second product's operands
      bf16x8_t first_v[T::D / 32];
      const int key0 = t * T::KT;
      if (key0 < see_lo || key0 + T::KT > see_hi) {
        asm volatile("");   // (a branch: few tiles lie on an edge)
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int key = key0 + 32 * u + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
            if (key < row_lo || key >= row_hi) sc[u][r] = -INFINITY;
          }
      }
      float top = sc[0][0];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[u][r]);
      const float most = fmaxf(mx, max_xor32(top) * scale2);
      if (__any(most > mx + kSlack)) {
        asm volatile("");
        const float f = __builtin_amdgcn_exp2f(mx - reference(most));
        mx = most;
        l *= f;
#pragma unroll
        for (int i = 0; i < T::D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[0][i][r] *= f;
      }
      const float ref = reference(mx) - kLift<C>;
      M::read_values(v0, 0, 0, lane, first_v);   // the first operands of the products
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          sc[u][r] = __builtin_amdgcn_exp2f(fmaf(sc[u][r], scale2, -ref));
          sum += sc[u][r];
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[u][ks][e] = pack_weights<C>(sc[u][8 * ks + 2 * e], sc[u][8 * ks + 2 * e + 1]);
      }
      l += sum;
      // (the probabilities belong to this phase)
#pragma unroll
      for (int x = 0; x < 2 * SUB; ++x)
        asm volatile("" : "+v"(pr[x / 2][x % 2].x), "+v"(pr[x / 2][x % 2].y), "+v"(pr[x / 2][x % 2].z),
                          "+v"(pr[x / 2][x % 2].w));
      __syncthreads();
      // ---- products: this tile's values, the next one's scores; and the copies between them.  In
      // every step the operands of the next are asked for, then the products of this one begun.
      if (stage.live != M::kAll) M::clear(tid, stage);
      __builtin_amdgcn_s_setprio(1);
      bool in;
      const uint64_t off = L::offset_of(p, page, in);
      const uint64_t live = __ballot(in) & M::kAll;
      u32x4_t k[2][T::QN];
#pragma unroll
      for (int x = 0; x < 2 * SUB; ++x) {
        bf16x8_t v[T::D / 32];
        if (x + 1 < 2 * SUB) M::read_values(v0, (x + 1) / 2, (x + 1) % 2, lane, v);
        else M::read_keys(k1, 0, lane, k[0]);
        if (x == 0) M::store_one(k2, tid, stage.k, std::true_type{});
        if (x == 1) M::store_one(v2, tid, stage.v, std::false_type{});
#pragma unroll
        for (int i = 0; i < T::D / 32; ++i)
          o[0][i] = weigh<C>(first_v[i], pr[x / 2][x % 2], o[0][i]);
#pragma unroll
        for (int i = 0; i < T::D / 32; ++i) first_v[i] = v[i];
        __builtin_amdgcn_sched_barrier(0);
      }
      // (past the last tile: keys and values that nobody reads)
      M::load_at(p, kb, vb, off, live, tid, stage);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        if (u + 1 < SUB) M::read_keys(k1, u + 1, lane, k[(u + 1) % 2]);
        if (u == 0) page = L::page_of(g, table, (t + 4) * T::KT, lo, hi, lane);
        f32x16_t c[1];
        M::scores(k[u % 2], q, c);
        sc[u] = c[0];
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      char* const k_old = k3;
      k3 = k1;
      k1 = k2;
      k2 = k_old;
      char* const v_old = v0;
      v0 = v1;
      v1 = v2;
      v2 = v3;
      v3 = v_old;
      __syncthreads();
    }
    if (wave < 4) __syncthreads();   // (the second four have one more behind them)
    l += __shfl_xor(l, 32);
    const float ms[1] = {mx}, ls[1] = {l};
    M::put_rows(g, s, h, m, wave * 32, lane, slot, o, ms, ls, v_scale);
    __syncthreads();   // the tiles in LDS are read: the next row tile may overwrite them
  }
};

// -------------------------------------------------------------- few rows
// 32-bit LDS address
__device__ __forceinline__ uint32_t lds_offset(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p));
}

// Transposing reads of four operands at LDS addresses a[i] + O0, a[i] + O1 (four 16-bit values of
// column lane % 16 from 4 rows x 16 columns each).  With its own wait: the compiler takes the
// intrinsic for a possible write to LDS and waits for the copies in flight before it.
template <int O0, int O1>
__device__ __forceinline__ void read_tr4(const uint32_t (&a)[4], bf16x8_t (&v)[4]) {
  i16x4_t l[4], h[4];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%c12\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:%c13\n\t"
      "ds_read_b64_tr_b16 %2, %9 offset:%c12\n\t"
      "ds_read_b64_tr_b16 %3, %9 offset:%c13\n\t"
      "ds_read_b64_tr_b16 %4, %10 offset:%c12\n\t"
      "ds_read_b64_tr_b16 %5, %10 offset:%c13\n\t"
      "ds_read_b64_tr_b16 %6, %11 offset:%c12\n\t"
      "ds_read_b64_tr_b16 %7, %11 offset:%c13\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(l[0]), "=&v"(h[0]), "=&v"(l[1]), "=&v"(h[1]), "=&v"(l[2]), "=&v"(h[2]), "=&v"(l[3]), "=&v"(h[3])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(O0), "n"(O1)
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = join_tr(l[i], h[i]);
}
// the same of e4m3: 8 codes of a column from 8 rows x 16 columns, widened
template <int O0>
__device__ __forceinline__ void read_tr4_codes(const uint32_t (&a)[4], bf16x8_t (&v)[4]) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  u32x2_t x[4];
  asm volatile(
      "ds_read_b64_tr_b8 %0, %4 offset:%c8\n\t"
      "ds_read_b64_tr_b8 %1, %5 offset:%c8\n\t"
      "ds_read_b64_tr_b8 %2, %6 offset:%c8\n\t"
      "ds_read_b64_tr_b8 %3, %7 offset:%c8\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(O0)
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = widen8_half(x[i].x, x[i].y);
}

static __device__ const uint32_t kZeros16[4] __attribute__((aligned(16))) = {0, 0, 0, 0};

// 16 bytes per lane, cache -> LDS: lane l's land at dst + 16 l (dst uniform).  Non-temporal: few
// rows read the cache once (16 x 8 rows over 16384 positions: 223 -> 204 us).
__device__ __forceinline__ void copy_lds16(const char* src, char* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 2);
}

template <typename T>
struct AttnFewBody : AttnLoader<T> {
  using L = AttnLoader<T>;
  using S = typename T::S;
  using C = typename T::C;

  // Where a tile's keys lie: from page ids that have arrived.
  struct Way {
    uint32_t lo, hi;   // this lane's key's bytes from the head's first
    uint64_t live;     // bit t: key t of the tile is read (others come from zeros)
  };
  static constexpr uint64_t kAll = T::KT == 64 ? ~0ull : 0xFFFFFFFFull;
  static __device__ __forceinline__ Way way(const AttnProblem& p, AttnPage a) {
    bool in;
    const uint64_t off = L::offset_of(p, a, in);
    return Way{static_cast<uint32_t>(off), static_cast<uint32_t>(off >> 32), __ballot(in) & kAll};
  }

  // Page ids of a tile to come, through LDS: a register would make the compiler wait for all loads
  // in flight, the last tile's values among them, where it is used.
  static __device__ __forceinline__ int32_t ask(const AttnArgs& g, const int32_t* table, int key0, int lo, int hi,
                                                int lane, char* ids) {
    int32_t place;
    const int32_t* at = table + L::column_of(g, key0, lo, hi, lane, place);
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)at,
                                     (__attribute__((address_space(3))) void*)ids, 4, 0, 0);
    return place;
  }
  static __device__ __forceinline__ AttnPage asked(const char* ids, int lane, int32_t place) {
    return AttnPage{*reinterpret_cast<const int32_t*>(ids + 4 * lane), place};
  }

  // A tile of keys or values on its way to LDS, LOADS loads.  Where all its keys are read and the
  // rows of a load lie in one page, the offset is the load's own scalar; else every lane takes its
  // row's, and keys that are not read come from zeros.  (turn: of a row's chunks in LDS.)
  template <typename Turn>
  static __device__ __forceinline__ void load(const AttnProblem& p, const char* base, const Way& w, int lane,
                                              char* to, Turn turn) {
    asm volatile("" : "+v"(lane));   // (offsets are made anew: held over the loop they take 4 LOADS registers)
    const uint32_t sub = lane / T::CPR, pos = lane % T::CPR;
    const uint32_t c = (pos ^ turn(sub)) << 4;   // (the turns of rows RPL i and sub are of different bits)
    if (w.live == kAll && L::whole_loads(p)) {
      const uint32_t mine = sub * p.token_bytes;
#pragma unroll
      for (int i = 0; i < T::LOADS; ++i) {
        const uint32_t l = __builtin_amdgcn_readlane(w.lo, T::RPL * i), h = __builtin_amdgcn_readlane(w.hi, T::RPL * i);
        const uint64_t at = (static_cast<uint64_t>(h) << 32) | l;
        copy_lds16(base + at + (mine + (c ^ (turn(T::RPL * i) << 4))), to + 1024 * i);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < T::LOADS; ++i) {
        const uint32_t row = T::RPL * i + sub;
        const uint32_t l = __shfl(static_cast<int>(w.lo), row), h = __shfl(static_cast<int>(w.hi), row);
        const uint64_t at = (static_cast<uint64_t>(h) << 32) | l;
        const char* zero = reinterpret_cast<const char*>(kZeros16);
        copy_lds16((w.live >> row) & 1 ? base + at + (c ^ (turn(T::RPL * i) << 4)) : zero, to + 1024 * i);
      }
    }
  }
  static __device__ __forceinline__ void load_keys(const AttnProblem& p, const char* kb, const Way& w, int lane, char* lk) {
    load(p, kb, w, lane, lk, [](uint32_t r) { return key_turn<T::ROWB>(r); });
  }
  static __device__ __forceinline__ void load_values(const AttnProblem& p, const char* vb, const Way& w, int lane, char* lv) {
    load(p, vb, w, lane, lv, [](uint32_t r) { return value_turn<T>(r); });
  }

  // first feature of query piece i of lane group grp: as the keys' operand takes them
  static __device__ __forceinline__ int q_place(int i, int grp) {
    if constexpr (T::CS == 1) return 64 * (i / 2) + 16 * grp + 8 * (i % 2);
    return (4 * i + grp) * (16 / T::ES);
  }

  // query piece i of row tile rt: a register, or LDS (as keys lie there)
  static __device__ __forceinline__ uint32_t q_lds(int row, int i, int grp) {
    return T::Q_AT + key_place<T::D * T::ES>(row, q_place(i, grp) * T::ES / 16);
  }

  // S^T of 32 keys against RT x 16 queries: pr[rt][4 u + r] of key 16 u + 4 (lane / 16) + r of query lane % 16
  static __device__ __forceinline__ void scores(const char* lds, const char* lk, int sub, int lane,
                                                const u32x4_t (&q)[T::RT][T::QLDS ? 1 : T::QN],
                                                float (&pr)[T::RT][8]) {
    f32x4_t c[2][T::RT];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt) c[u][rt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto query = [&](int rt, int i) -> u32x4_t {
      if constexpr (T::QLDS) return load16(lds + q_lds(16 * rt + (lane & 15), i, lane >> 4));
      else return q[rt][i];
    };
    const uint32_t row = 32 * sub + (lane & 15);
#pragma unroll
    for (int i = 0; i < T::ROWB / 64; ++i) {
      u32x4_t a[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) a[u] = load16(lk + key_place<T::ROWB>(row + 16 * u, 4 * i + (lane >> 4)));
      if constexpr (T::CS == 1) {
        u32x4_t x[2], y[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) widen16(a[u], x[u], y[u]);
#pragma unroll
        for (int rt = 0; rt < T::RT; ++rt) {
          const u32x4_t q0 = query(rt, 2 * i), q1 = query(rt, 2 * i + 1);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            c[u][rt] = mma16(x[u], q0, c[u][rt], S{});
            c[u][rt] = mma16(y[u], q1, c[u][rt], S{});
          }
        }
      } else {
#pragma unroll
        for (int rt = 0; rt < T::RT; ++rt) {
          const u32x4_t q0 = query(rt, i);
#pragma unroll
          for (int u = 0; u < 2; ++u) c[u][rt] = mma16(a[u], q0, c[u][rt], S{});
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt)
#pragma unroll
      for (int i = 0; i < 8; ++i) pr[rt][i] = c[i / 4][rt][i % 4];
  }

  // O^T += V^T P^T of 32 keys: features 16 i + 4 (lane / 16) + r of query lane % 16.  A lane's
  // probabilities pr[0 .. 4) are of keys 4 (lane / 16) + r, pr[4 .. 8) of those plus 16.
  static __device__ __forceinline__ void add_values(const char* lv, int sub, int lane,
                                                    const float (&pr)[T::RT][8],
                                                    f32x4_t (&o)[T::RT][T::D / 16]) {
    const int grp = lane >> 4;
    if constexpr (T::ES == 2) {
      u32x4_t b[T::TERMS][T::RT];
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = pr[rt][2 * e], y = pr[rt][2 * e + 1];
          if constexpr (T::TERMS == 2) {
            const uint2 w = split_weights(x, y);
            b[0][rt][e] = w.x;
            b[1][rt][e] = w.y;
          } else {
            b[0][rt][e] = pack_weights<C>(x, y);
          }
        }
      // 8 bytes of row `row` (and of 16 rows on) per lane; the turns of the chunks 2 i (i, e4m3) and
      // of the lane's own are of different bits
      const uint32_t e = (lane & 15) >> 1;
      const uint32_t row = T::CS == 2 ? 4 * grp + ((lane & 15) >> 2) : 4 * grp + (e & 3) + 4 * (e & 4);
      const uint32_t at = lds_offset(lv) + value_place<T>(row, T::CS == 2 ? (lane >> 1) & 1 : 0) + (lane & 1) * 8;
#pragma unroll
      for (int i0 = 0; i0 < T::D / 16; i0 += 4) {
        uint32_t ad[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ad[i] = at ^ ((i0 + i) * 16 * T::CS);
        bf16x8_t a[4];
        if constexpr (T::CS == 2) {
          if (sub == 0) read_tr4<0, 16 * T::ROWB>(ad, a);
          else read_tr4<32 * T::ROWB, 48 * T::ROWB>(ad, a);
        } else {
          if (sub == 0) read_tr4_codes<0>(ad, a);
          else read_tr4_codes<32 * T::ROWB>(ad, a);
        }
#pragma unroll
        for (int x = 0; x < T::TERMS; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int rt = 0; rt < T::RT; ++rt)
              o[rt][i0 + i] = weigh<C>(a[i], b[x][rt], o[rt][i0 + i]);
      }
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint32_t row = 32 * sub + 16 * (x / 4) + 4 * grp + x % 4;
#pragma unroll
        for (int i = 0; i < T::D / 16; ++i) {
          const uint32_t d = 16 * i + (lane & 15);
          const float a = *reinterpret_cast<const float*>(lv + value_place<T>(row, d / 4) + (d & 3) * 4);
#pragma unroll
          for (int rt = 0; rt < T::RT; ++rt)
            o[rt][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, pr[rt][x], o[rt][i], 0, 0, 0);
        }
      }
    }
  }

  static __device__ __forceinline__ void run(const AttnArgs& g, const AttnSeq& s, int b, int h, int m, int ta,
                                             int tb, int lo, int hi, int64_t slot, char* lds) {
    const AttnProblem& p = g.p;
    const int wn = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int r0 = m * T::BM;
    const int rows = s.n * p.group;
    float scale2 = g.scale2, v_scale = 1.f;
    if constexpr (sizeof(C) == 1) {
      scale2 *= p.k_scale[h];
      v_scale = p.v_scale[h];
    }
    const AttnSign sign = positive<C>(scale2);

    const int32_t* table = p.table + static_cast<int64_t>(b) * p.width;
    const char* kb = static_cast<const char*>(p.k_cache) + h * p.head_bytes;
    const char* vb = static_cast<const char*>(p.v_cache) + h * p.head_bytes;
    char* const base = lds + wn * T::WAVE_BYTES;
    char* lk = base;
    char* lv = lk + T::TILE_BYTES;
    char* other = base + 2 * T::TILE_BYTES;   // (two tiles)
    // A tile's loads: its keys', the page ids of the tile after it, its values'.  They return in
    // that order, so what is in flight tells what has arrived.
    int t = ta + wn;
    Way w{};
    char* const ids = lds + T::PAGE_AT + 256 * wn;
    int32_t place = 0;
    if (t < tb) {
      w = way(p, L::page_of(g, table, t * T::KT, lo, hi, lane));
      load_keys(p, kb, w, lane, lk);
      __builtin_amdgcn_sched_barrier(0);   // (the order that the waits count on)
      place = ask(g, table, (t + T::WN) * T::KT, lo, hi, lane, ids);
      __builtin_amdgcn_sched_barrier(0);
      load_values(p, vb, w, lane, lv);
    }
    u32x4_t q[T::RT][T::QLDS ? 1 : T::QN];
    int row_lo[T::RT], row_hi[T::RT];
    f32x4_t o[T::RT][T::D / 16];
    float mx[T::RT], l[T::RT];
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) {
      const int r = r0 + 16 * rt + (lane & 15);
      if constexpr (T::QLDS) {
        if (wn == rt) {   // (WN waves, a row tile each: RT <= WN)
          u32x4_t x[T::QN];
          L::load_q(p, s, h, r, [&](int i) { return q_place(i, lane >> 4); }, sign, x);
#pragma unroll
          for (int i = 0; i < T::QN; ++i)
            *reinterpret_cast<u32x4_t*>(lds + q_lds(16 * rt + (lane & 15), i, lane >> 4)) = x[i];
        }
      } else {
        L::load_q(p, s, h, r, [&](int i) { return q_place(i, lane >> 4); }, sign, q[rt]);
      }
      const int at = s.len - s.n + r / p.group;
      row_hi[rt] = p.causal ? min(at + 1, s.len) : s.len;
      row_lo[rt] = p.window ? at - p.window + 1 : 0;
      mx[rt] = -INFINITY;
      l[rt] = 0.f;
#pragma unroll
      for (int i = 0; i < T::D / 16; ++i) o[rt][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // the rows all see the keys [see_lo, see_hi)
    const int first = s.len - s.n + r0 / p.group;
    const int last = s.len - s.n + min(r0 + T::BM - 1, rows - 1) / p.group;
    const int see_hi = p.causal ? min(first + 1, s.len) : s.len;
    const int see_lo = p.window ? last - p.window + 1 : 0;

    if constexpr (T::QLDS) __syncthreads();   // the queries are in LDS
    for (; t < tb; t += T::WN) {
      // The wave's own LDS: it waits for its own loads only.  Keys (and page ids) are there when the
      // values' loads alone are in flight.
      asm volatile("" ::: "memory");
      BDR_WAIT_VM(T::LOADS);
      asm volatile("" ::: "memory");
      const int key0 = t * T::KT;
      const bool edge = key0 < see_lo || key0 + T::KT > see_hi;
      const bool more = t + T::WN < tb;
      if constexpr (T::BUFS == 2) {
        const AttnPage page = asked(ids, lane, place);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (more) {
          w = way(p, page);
          load_keys(p, kb, w, lane, other);
          __builtin_amdgcn_sched_barrier(0);   // (the order that the waits count on)
          place = ask(g, table, (t + 2 * T::WN) * T::KT, lo, hi, lane, ids);
          __builtin_amdgcn_sched_barrier(0);
          load_values(p, vb, w, lane, other + T::TILE_BYTES);
        }
      }
      float pr[T::KT / 32][T::RT][8];
#pragma unroll
      for (int u = 0; u < T::KT / 32; ++u) scores(lds, lk, u, lane, q, pr[u]);
      if constexpr (T::BUFS == 1) {
        const AttnPage page = asked(ids, lane, place);
        // every read of the keys and ids has returned: the next tile's take their place
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (more) {
          w = way(p, page);
          load_keys(p, kb, w, lane, lk);
          __builtin_amdgcn_sched_barrier(0);
          place = ask(g, table, (t + 2 * T::WN) * T::KT, lo, hi, lane, ids);
        }
      }
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt) {
        float z[T::KT / 4];
#pragma unroll
        for (int i = 0; i < T::KT / 4; ++i) z[i] = pr[i / 8][rt][i % 8];
        const float was = mx[rt];
        const float f = softmax_step<C, T::KT / 4>(
            z, edge, row_lo[rt], row_hi[rt], scale2,
            [&](int i) { return key0 + 16 * (i / 4) + 4 * (lane >> 4) + i % 4; },
            [](float v) { return max_xor32(max_xor16(v)); }, mx[rt], l[rt]);
        if (__any(mx[rt] > was)) {
          asm volatile("");
#pragma unroll
          for (int i = 0; i < T::D / 16; ++i) o[rt][i] *= f;
        }
#pragma unroll
        for (int i = 0; i < T::KT / 4; ++i) pr[i / 8][rt][i % 8] = z[i];
      }
      // values: what is in flight behind them are the next keys and page ids (and values)
      asm volatile("" ::: "memory");
      if (more) BDR_WAIT_VM(T::LOADS * T::BUFS + 1);
      else BDR_WAIT_VM(0);
      asm volatile("" ::: "memory");
#pragma unroll
      for (int u = 0; u < T::KT / 32; ++u) add_values(lv, u, lane, pr[u], o);
      // every read of the values has returned
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (T::BUFS == 1) {
        if (more) load_values(p, vb, w, lane, lv);
      } else {
        char* const last = lk;
        lk = other;
        lv = other + T::TILE_BYTES;
        other = last;
      }
    }
    lk = base;

    // join the waves' states through LDS, 16 rows at a time
    auto ml = [&](int w) { return reinterpret_cast<float2*>(lds + w * T::WAVE_BYTES + 16 * T::D * 4); };
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) {
      const int qi = lane & 15;
      l[rt] += __shfl_xor(l[rt], 16);
      l[rt] += __shfl_xor(l[rt], 32);
#pragma unroll
      for (int i = 0; i < T::D / 16; ++i) {
        const uint32_t c = 4 * i + (lane >> 4);   // 16-byte chunk of the row
        *reinterpret_cast<f32x4_t*>(lk + qi * T::D * 4 + ((c ^ qi) << 4)) = o[rt][i];
      }
      if (lane < 16) ml(wn)[qi] = float2{mx[rt], l[rt]};
      __syncthreads();
      for (int idx = static_cast<int>(threadIdx.x); idx < 16 * (T::D / 4); idx += T::THREADS) {
        const int qr = idx / (T::D / 4), c = idx % (T::D / 4);
        const int rl = 16 * rt + qr;
        const int r = r0 + rl;
        if (r < rows) {
          float mm = ml(0)[qr].x;
#pragma unroll
          for (int w = 1; w < T::WN; ++w) mm = fmaxf(mm, ml(w)[qr].x);
          const float ref = mm == -INFINITY ? 0.f : mm;
          float ls = 0.f;
          f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < T::WN; ++w) {
            const float f = __builtin_amdgcn_exp2f(ml(w)[qr].x - ref);
            ls += f * ml(w)[qr].y;
            v += f * *reinterpret_cast<const f32x4_t*>(lds + w * T::WAVE_BYTES + qr * T::D * 4 + ((c ^ qr) << 4));
          }
          if (slot >= 0) {
            *reinterpret_cast<f32x4_t*>(g.part_o + (slot * T::BM + rl) * T::D + 4 * c) = v;
            if (c == 0) g.part_ml[slot * T::BM + rl] = float2{mm, ls};
          } else {
            L::put(g, s.first, h, r, 4 * c, v, mm, ls, v_scale);
          }
        }
      }
      __syncthreads();
    }
  }
};

template <typename T>
using AttnBody =
    std::conditional_t<T::kFew, AttnFewBody<T>, std::conditional_t<T::kTall, AttnTallBody<T>, AttnManyBody<T>>>;

// The workgroup's share of one kv head's key tiles, row tile by row tile.
template <typename T>
__global__ __launch_bounds__(T::THREADS, T::SIMD_WAVES) void attn_kernel(const AttnArgs g) {
  using Plan = AttnPlan<T::BM, T::KT>;
  __shared__ __attribute__((aligned(16))) char lds[T::LDS_BYTES];
  const AttnProblem& p = g.p;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  // every wave sums and searches for itself: no barriers
  int64_t all = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    const int b = b0 + lane;
    all += b < p.batch ? Plan::total(Plan::seq(p, g.whole, b)) : 0;
  }
  all = uniform_i64(wave_sum_i64(all));
  const int64_t share = g.whole ? 1 : max(g.min_share, (all + g.shares - 1) / g.shares);
  // Share w of kv head h.  Few rows: the heads of a share side by side.  Many rows: neighbours read
  // the same keys, so where every workgroup has work a head's neighbours go to one XCD (workgroups
  // go round the eight) and its L2 (4 x 1024 tokens over 8192 bf16 keys of 128: 292 -> 278 us).
  int h = static_cast<int>(blockIdx.x) % p.hkv;
  int64_t w = static_cast<int>(blockIdx.x) / p.hkv;
  if (!T::kFew && share > g.min_share && gridDim.x % 8 == 0) {
    const uint32_t i = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8, shares = gridDim.x / p.hkv;
    h = static_cast<int>(i / shares);
    w = i % shares;
  }
  const int64_t id = w * p.hkv + h;
  int64_t x = w * share;
  const int64_t end = min(x + share, all);
  int32_t* const rec = g.record + id * kRecord;
  if (threadIdx.x == 0 && !g.whole) rec[3] = -1;
  if (x >= end) return;
  // the request that holds x
  int b = 0;
  int64_t base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    const int bl = b0 + lane;
    const int64_t own = bl < p.batch ? Plan::total(Plan::seq(p, g.whole, bl)) : 0;
    int64_t c = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t u = __shfl_up(c, d);
      if (lane >= d) c += u;
    }
    const uint64_t past = __ballot(base + c > x);
    if (past) {
      const int at = __ffsll(static_cast<long long>(past)) - 1;
      b = b0 + at;
      base = uniform_i64(base + __shfl(c - own, at));
      break;
    }
    base = uniform_i64(base + __shfl(c, 63));
  }
  b = __builtin_amdgcn_readfirstlane(b);
  AttnSeq s = Plan::seq(p, g.whole, b);
  int u = static_cast<int>((x - base) / s.cost);
  int inner = static_cast<int>(x - base - static_cast<int64_t>(u) * s.cost);
  while (x < end) {
    // the unit's row tiles: the longer, then (paired) the shorter
    int done = 0;
    for (int part = 0; part < 2 && x < end; ++part) {
      const int m = s.paired && part == 0 ? s.tiles - 1 - u : u;
      if (part == 1 && (!s.paired || u == s.tiles - 1 - u)) break;
      int lo, hi, t0, t1;
      Plan::range(p, s, m, lo, hi, t0, t1);
      const int nt = t1 - t0;
      if (inner < done + nt) {
        const int from = g.whole ? 0 : inner - done;
        const int to = g.whole ? nt : static_cast<int>(min(static_cast<int64_t>(nt), from + (end - x)));
        int64_t slot = -1;   // of a partial: what the workgroup before began, or what the next goes on with
        if (from > 0) {
          slot = 2 * id;
          if (threadIdx.x == 0) {
            // x0 is where the row tile begins; the first border inside it does the join
            const int64_t x0 = x - from;
            rec[0] = s.first;
            rec[1] = s.n;
            rec[2] = m;
            rec[3] = x0 / share == w - 1 ? static_cast<int32_t>((x0 + nt - 1) / share) : -1;
          }
        } else if (to < nt) {
          slot = 2 * id + 1;
        }
        AttnBody<T>::run(g, s, b, h, m, t0 + from, t0 + to, lo, hi, slot, lds);
        if (g.whole) return;
        x += to - from;
        inner += to - from;
      }
      done += nt;
    }
    if (x >= end) break;
    x += s.cost - inner;   // what the unit costs less than its request's units at most
    inner = 0;
    if (++u == s.units) {
      u = 0;
      do {
        if (++b >= p.batch) return;
        s = Plan::seq(p, g.whole, b);
      } while (s.units == 0);
    }
  }
}

// Joins the partials of the row tiles that several workgroups share: blockIdx.x + hkv is
// the id of the workgroup whose share begins inside one, blockIdx.y the rows.
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs g) {
  const AttnProblem& p = g.p;
  const int h = static_cast<int>(blockIdx.x) % p.hkv;
  const int w = static_cast<int>(blockIdx.x) / p.hkv + 1;
  const int32_t* rec = g.record + static_cast<int64_t>(blockIdx.x + p.hkv) * kRecord;
  const int last = rec[3];
  if (last < 0) return;
  const int first = rec[0], rows = rec[1] * p.group, m = rec[2];
  float v_scale = 1.f;
  if constexpr (sizeof(typename T::C) == 1) v_scale = p.v_scale[h];
  constexpr int PER = 256 / (T::D / 4);   // rows of a workgroup
  constexpr int AHEAD = 8;                // partials asked for together: their latency bounds this
  const int c = static_cast<int>(threadIdx.x) % (T::D / 4);
  for (int rl = blockIdx.y * PER + static_cast<int>(threadIdx.x) / (T::D / 4);
       rl < T::BM && m * T::BM + rl < rows; rl += PER * static_cast<int>(gridDim.y)) {
    const int r = m * T::BM + rl;
    float mm = -INFINITY, l = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = w - 1; i0 <= last; i0 += AHEAD) {
      float2 ml[AHEAD];
      f32x4_t part[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int at = min(i0 + i, last);
        const int64_t slot = (2 * (static_cast<int64_t>(at) * p.hkv + h) + (at == w - 1 ? 1 : 0)) * T::BM + rl;
        ml[i] = g.part_ml[slot];
        part[i] = *reinterpret_cast<const f32x4_t*>(g.part_o + slot * T::D + 4 * c);
      }
      float top = mm;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (i0 + i > last) ml[i] = float2{-INFINITY, 0.f};
        top = fmaxf(top, ml[i].x);
      }
      const float ref = top == -INFINITY ? 0.f : top;
      const float f0 = __builtin_amdgcn_exp2f(mm - ref);
      l *= f0;
      o *= f0;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const float f = __builtin_amdgcn_exp2f(ml[i].x - ref);
        l += f * ml[i].y;
        if (i0 + i <= last) o += f * part[i];
      }
      mm = top;
    }
    AttnLoader<T>::put(g, first, h, r, 4 * c, o, mm, l, v_scale);
  }
}

}  // namespace bdr
