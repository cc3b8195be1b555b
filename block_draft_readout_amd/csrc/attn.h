// Attention of new tokens over a paged cache (gfx950): types, schedule and kernel.
//
//   out[q] = sum_t softmax_t(scale q . k[t]) v[t]  over the positions t that the
//   token sees, in one pass with a running maximum m and sum l: a tile of keys
//   gives S = K Q^T, m' = max(m, max S), P = 2^(S - m'), and
//   O = O 2^(m - m') + V^T P,  l = l 2^(m - m') + sum P;  out = O / l.
//
// Work.  The query heads that share a kv head read the same keys, so request b's
// n tokens and the `group` heads of a kv head are packed into n * group rows, BM
// of which make a row tile.  A row tile walks its visible keys in tiles of KT.
// Lengths live on the device and differ widely, so the launch has a fixed number
// of workgroups and each takes an equal, contiguous share of all key tiles of all
// (request, kv head, row tile): it finds its place from the lengths by a prefix
// sum.  A row tile that ends up with several workgroups gets partial (O, m, l) in
// the workspace, which a second launch joins in order: nothing depends on the
// order of arrival.
//
// Products.  S is computed transposed (keys are the rows of the MFMA's result), so
// a lane holds one query's column: its maximum, sum and rescaling are the lane's
// own, and the 32 x 32 result's registers are, rounded to bf16, the operand of the
// second product as they lie (the keys of a step are taken in the order in which
// a lane's registers hold them; V is read with the same order).
#pragma once

#include "train_device.h"

namespace bdr {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));

struct AttnArgs {
  AttnProblem p;
  int64_t slabs;        // workgroups of the schedule
  int64_t min_share;    // key tiles that a workgroup takes at least
  int whole;            // each row tile is one workgroup's
  float scale2;         // scale * log2(e)
  float* part_o;        // [2 * slabs][BM][D]
  float2* part_ml;      // [2 * slabs][BM] (m in units of log2, l)
  int32_t* record;      // [slabs][kRecord] what the join needs
};

constexpr int kRecord = 8;   // first row, tokens, kv head, row tile, last workgroup (-1: nothing to join)

// -------------------------------------------------------------- schedule
// A request: its rows, row tiles and what they cost in key tiles.  A unit is a row
// tile, or, where causal row tiles differ much, a long and a short one together:
// every unit of a request then costs the same, at most `cost`.
struct AttnSeq {
  int32_t first, n, len;
  int32_t tiles;    // row tiles
  int32_t units;    // per kv head
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
  static __device__ __forceinline__ int64_t total(const AttnProblem& p, const AttnSeq& s) {
    return static_cast<int64_t>(p.hkv) * s.units * s.cost;
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
template <typename C_, typename S_, int D_, int WM_, int WN_, int RT_, int KT_>
struct AttnTile {
  using C = C_;                       // cache element: uint16_t (bf16), uint8_t (e4m3) or float
  using S = S_;                       // queries, output and LDS: uint16_t or float
  static constexpr int D = D_;
  // WM waves hold different rows and share their keys' tiles in LDS, or (WM = 1) WN
  // waves hold the same rows and walk key tiles of their own, joined at the end
  static constexpr int WM = WM_, WN = WN_;
  static constexpr int RT = RT_;      // 32-row tiles of a wave
  static constexpr int KT = KT_;      // keys of a tile
  static constexpr int THREADS = 64 * WM * WN;
  static constexpr int BM = 32 * WM * RT;
  static constexpr int ES = static_cast<int>(sizeof(S));
  static constexpr int ROWB = D * ES;                    // bytes of an LDS row
  static constexpr int PER16 = 16 / static_cast<int>(sizeof(C));   // cache elements of 16 bytes
  static constexpr int CPR = D / PER16;                  // 16-byte pieces of a cache row
  static constexpr int SHARE = 64 * WM;                  // threads that load a tile
  static constexpr int LOADS = KT * CPR / SHARE;         // 16-byte loads of a thread, K or V
  static constexpr int TILE_BYTES = KT * ROWB;           // K or V of a tile
  static constexpr int BUFS = WM > 1 ? 2 : 1;
  static constexpr int JOIN_BYTES = WN > 1 ? 32 * D * 4 : 0;   // a wave's O of 32 rows
  static constexpr int WAVE_BYTES = std::max(2 * TILE_BYTES * BUFS, JOIN_BYTES);
  static constexpr int LDS_BYTES = WAVE_BYTES * WN;
  static constexpr int QN = ROWB / 32;                   // 16-byte query pieces of a lane and row
  static_assert(WM == 1 || WN == 1, "rows or keys are split over the waves");
  static_assert(KT % 32 == 0 && KT <= 64, "a lane looks up one key's page");
  static_assert(LOADS * SHARE == KT * CPR, "loads split evenly");
  static_assert(LDS_BYTES <= 160 * 1024, "tile fits");
};

// Places of the 16-byte chunks c of LDS row r, so that 16 lanes that read a chunk of 16
// rows (keys), and 32 lanes that read 64 bytes of 4 rows (values), meet distinct banks.
template <int ROWB>
__device__ __forceinline__ uint32_t key_place(uint32_t r, uint32_t c) {
  const uint32_t x = ROWB >= 256 ? r & 15u : (r >> 1) & 7u;
  return r * ROWB + ((c ^ x) << 4);
}
template <int ROWB>
__device__ __forceinline__ uint32_t value_place(uint32_t r, uint32_t c) {
  const uint32_t x = ROWB >= 256 ? (r & 3u) << 2 : (r & 2u) << 1;
  return r * ROWB + ((c ^ x) << 4);
}

// 16 e4m3 codes as bf16 (every code's value is one)
__device__ __forceinline__ void widen16(u32x4_t v, u32x4_t& a, u32x4_t& b) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, false);
    const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, true);
    const uint32_t l = __builtin_bit_cast(uint32_t, lo), h = __builtin_bit_cast(uint32_t, hi);
    if (i < 2) {
      a[2 * i] = l;
      a[2 * i + 1] = h;
    } else {
      b[2 * (i - 2)] = l;
      b[2 * (i - 2) + 1] = h;
    }
  }
}

template <typename T>
struct AttnState {
  f32x16_t o[T::RT][T::D / 32];   // O^T: features 32 i + 8 (r / 4) + 4 (lane / 32) + r % 4 of query lane % 32
  float m[T::RT], l[T::RT];       // running maximum (units of log2), this half wave's sum
};

// A staged tile: what a thread holds of the next keys and values.
template <typename T>
struct AttnStage {
  u32x4_t k[T::LOADS], v[T::LOADS];
  uint64_t live;                  // bit t: key t of the tile is read (others are zeros)
};

template <typename T>
struct AttnBody {
  using S = typename T::S;
  using C = typename T::C;
  using Plan = AttnPlan<T::BM, T::KT>;

  // where key t of a tile lies in the cache (elements from the head's base), and whether it is read
  static __device__ __forceinline__ void look_up(const AttnProblem& p, const int32_t* table, int key0,
                                                 int lo, int hi, int lane, int64_t& off, uint64_t& live) {
    const int key = key0 + (T::KT == 64 ? lane : lane & 31);
    bool in = key >= lo && key < hi;
    off = 0;
    if (in) {
      const uint32_t col = static_cast<uint32_t>(key) / static_cast<uint32_t>(p.page);
      const int32_t page = table[col];
      in = page >= 0 && page < p.pages;
      if (in)
        off = page * p.page_stride + (static_cast<uint32_t>(key) - col * p.page) * p.token_stride;
    }
    live = __ballot(in);
  }

  static __device__ __forceinline__ void load(const C* kb, const C* vb, int64_t off, uint64_t live, int st,
                                              AttnStage<T>& g) {
    const int lo = static_cast<int>(off), hi = static_cast<int>(off >> 32);
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
      const int idx = st + T::SHARE * i;
      const int row = idx / T::CPR, c = idx % T::CPR;
      const uint32_t l = __shfl(lo, row), h = __shfl(hi, row);
      // a key that is not read takes the first page's first row, and is cleared below
      const int64_t at = static_cast<int64_t>((static_cast<uint64_t>(h) << 32) | l) + c * T::PER16;
      g.k[i] = load16(kb + at);
      g.v[i] = load16(vb + at);
    }
    g.live = live;
  }

  static __device__ __forceinline__ void store(char* lk, char* lv, int st, AttnStage<T>& g) {
    constexpr uint64_t kAll = T::KT == 64 ? ~0ull : 0xFFFFFFFFull;
    const bool clear = (g.live & kAll) != kAll;
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
      const int idx = st + T::SHARE * i;
      const int row = idx / T::CPR, c = idx % T::CPR;
      u32x4_t k = g.k[i], v = g.v[i];
      if (clear && !((g.live >> row) & 1)) k = v = u32x4_t{0, 0, 0, 0};
      if constexpr (sizeof(C) == 1) {
        u32x4_t a, b;
        widen16(k, a, b);
        *reinterpret_cast<u32x4_t*>(lk + key_place<T::ROWB>(row, 2 * c)) = a;
        *reinterpret_cast<u32x4_t*>(lk + key_place<T::ROWB>(row, 2 * c + 1)) = b;
        widen16(v, a, b);
        *reinterpret_cast<u32x4_t*>(lv + value_place<T::ROWB>(row, 2 * c)) = a;
        *reinterpret_cast<u32x4_t*>(lv + value_place<T::ROWB>(row, 2 * c + 1)) = b;
      } else {
        *reinterpret_cast<u32x4_t*>(lk + key_place<T::ROWB>(row, c)) = k;
        *reinterpret_cast<u32x4_t*>(lv + value_place<T::ROWB>(row, c)) = v;
      }
    }
  }

  // 16-byte pieces of a row tile's queries: piece s of a lane is chunk 2 s + lane / 32 of query lane % 32
  static __device__ __forceinline__ void load_q(const AttnProblem& p, const AttnSeq& s, int h, int r0,
                                                int lane, bool flip, u32x4_t (&q)[T::QN]) {
    const int r = r0 + (lane & 31);
    const bool in = r < s.n * p.group;
    const int j = in ? r / p.group : 0;
    const int head = in ? h * p.group + (r - j * p.group) : 0;
    const S* at = static_cast<const S*>(p.q) + static_cast<int64_t>(s.first + j) * p.q_row +
                  static_cast<int64_t>(head) * p.q_head + (lane >> 5) * (16 / T::ES);
    const uint32_t sign = flip ? (T::ES == 2 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
    for (int i = 0; i < T::QN; ++i) {
      const u32x4_t v = in ? load16(at + i * (32 / T::ES)) : u32x4_t{0, 0, 0, 0};
      q[i] = u32x4_t{v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign};
    }
  }

  // S^T of 32 keys against 32 queries
  static __device__ __forceinline__ f32x16_t scores(const char* lk, int sub, int lane,
                                                    const u32x4_t (&q)[T::QN]) {
    f32x16_t c = {};
    const uint32_t row = 32 * sub + (lane & 31);
#pragma unroll
    for (int i = 0; i < T::QN; ++i) {
      const u32x4_t a = load16(lk + key_place<T::ROWB>(row, 2 * i + (lane >> 5)));
      if constexpr (T::ES == 2) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                    __builtin_bit_cast(bf16x8_t, q[i]), c, 0, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(q[i][e]), c, 0, 0, 0);
      }
    }
    return c;
  }

  // O^T += V^T P^T of 32 keys, whose probabilities a lane holds as the scores' registers lie
  static __device__ __forceinline__ void add_values(const char* lv, int sub, int lane,
                                                    const f32x16_t (&p)[T::RT], AttnState<T>& st) {
    const int half = lane >> 5;
    if constexpr (T::ES == 2) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4_t b[T::RT];
#pragma unroll
        for (int rt = 0; rt < T::RT; ++rt)
#pragma unroll
          for (int e = 0; e < 4; ++e) b[rt][e] = pack_bf16(p[rt][8 * ks + 2 * e], p[rt][8 * ks + 2 * e + 1]);
        // lanes of a group of 16 read 4 keys x 16 features, each 8 bytes, and get a column of it
        const uint32_t row = 32 * sub + 16 * ks + 4 * half + ((lane & 15) >> 2);
#pragma unroll
        for (int i = 0; i < T::D / 32; ++i) {
          const uint32_t c = 4 * i + ((lane >> 3) & 2) + ((lane >> 1) & 1);
          typedef __attribute__((address_space(3))) i16x4_t* lds_t;
          const i16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_t)(lv + value_place<T::ROWB>(row, c) + (lane & 1) * 8));
          const i16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_t)(lv + value_place<T::ROWB>(row + 8, c) + (lane & 1) * 8));
          typedef short i16x8_t __attribute__((ext_vector_type(8)));
          const i16x8_t a = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int rt = 0; rt < T::RT; ++rt)
            st.o[rt][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b[rt]), st.o[rt][i], 0, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t row = 32 * sub + 8 * (r / 4) + 4 * half + r % 4;
#pragma unroll
        for (int i = 0; i < T::D / 32; ++i) {
          const uint32_t d = 32 * i + (lane & 31);
          const float a = *reinterpret_cast<const float*>(lv + value_place<T::ROWB>(row, d / 4) + (d & 3) * 4);
#pragma unroll
          for (int rt = 0; rt < T::RT; ++rt)
            st.o[rt][i] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, p[rt][r], st.o[rt][i], 0, 0, 0);
        }
      }
    }
  }

  // One tile of keys [key0, key0 + KT): row_lo / row_hi bound what a lane's query sees; `edge`
  // where some query of the wave does not see all of it.
  static __device__ __forceinline__ void tile(const char* lk, const char* lv, int key0, int lane, bool edge,
                                              float scale2, const u32x4_t (&q)[T::RT][T::QN],
                                              const int (&row_lo)[T::RT], const int (&row_hi)[T::RT],
                                              AttnState<T>& st) {
    constexpr int SUB = T::KT / 32;
    f32x16_t s[SUB][T::RT];
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt) s[u][rt] = scores(lk, u, lane, q[rt]);
    if (edge) {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = key0 + 32 * u + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
#pragma unroll
          for (int rt = 0; rt < T::RT; ++rt)
            if (key < row_lo[rt] || key >= row_hi[rt]) s[u][rt][r] = -INFINITY;
        }
    }
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) {
      float top = s[0][rt][0];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][rt][r]);
      top = fmaxf(top, __shfl_xor(top, 32));   // the other half wave holds the other keys
      const float m = fmaxf(st.m[rt], top * scale2);
      if (__any(m > st.m[rt])) {
        const float f = __builtin_amdgcn_exp2f(st.m[rt] - (m == -INFINITY ? 0.f : m));
        st.l[rt] *= f;
#pragma unroll
        for (int i = 0; i < T::D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) st.o[rt][i][r] *= f;
        st.m[rt] = m;
      }
      const float ref = m == -INFINITY ? 0.f : m;   // (nothing seen yet)
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float e = __builtin_amdgcn_exp2f(fmaf(s[u][rt][r], scale2, -ref));
          s[u][rt][r] = e;
          sum += e;
        }
      st.l[rt] += sum;
    }
#pragma unroll
    for (int u = 0; u < SUB; ++u) add_values(lv, u, lane, s[u], st);
  }

  // rows of the output: out = o / l, or a partial
  static __device__ __forceinline__ void put(const AttnArgs& g, const AttnSeq& s, int h, int r, int d,
                                             f32x4_t o, float m, float l, float v_scale) {
    const AttnProblem& p = g.p;
    const int j = r / p.group;
    const int head = h * p.group + (r - j * p.group);
    const int64_t row = (static_cast<int64_t>(s.first) + j) * p.hq + head;
    const float inv = l > 0.f ? v_scale / l : 0.f;
    S* out = static_cast<S*>(p.out) + row * T::D + d;
    if constexpr (T::ES == 2)
      *reinterpret_cast<uint2*>(out) = uint2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
    else
      *reinterpret_cast<f32x4_t*>(out) = f32x4_t{o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
    if (p.lse && d == 0) p.lse[row] = l > 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
  }

  // One row tile over key tiles [ta, tb).  slot < 0: the output itself, else a partial there.
  static __device__ __forceinline__ void run(const AttnArgs& g, const AttnSeq& s, int b, int h, int m, int ta,
                                             int tb, int lo, int hi, int64_t slot, char* lds) {
    const AttnProblem& p = g.p;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int wm = T::WM > 1 ? wave : 0, wn = T::WM > 1 ? 0 : wave;
    const int st_id = T::WM > 1 ? static_cast<int>(threadIdx.x) : lane;   // place among the loading threads
    const int r0 = m * T::BM + wm * 32 * T::RT;
    const int rows = s.n * p.group;
    float scale2 = g.scale2, v_scale = 1.f;
    if constexpr (sizeof(C) == 1) {
      scale2 *= p.k_scale[h];
      v_scale = p.v_scale[h];
    }
    const bool flip = scale2 < 0.f;   // the running maximum wants a positive scale
    scale2 = fmaxf(fabsf(scale2), 1e-30f);

    u32x4_t q[T::RT][T::QN];
    int row_lo[T::RT], row_hi[T::RT];
    AttnState<T> st;
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) {
      load_q(p, s, h, r0 + 32 * rt, lane, flip, q[rt]);
      const int at = s.len - s.n + (r0 + 32 * rt + (lane & 31)) / p.group;
      row_hi[rt] = p.causal ? min(at + 1, s.len) : s.len;
      row_lo[rt] = p.window ? at - p.window + 1 : 0;
      st.m[rt] = -INFINITY;
      st.l[rt] = 0.f;
#pragma unroll
      for (int i = 0; i < T::D / 32; ++i) st.o[rt][i] = f32x16_t{};
    }
    // the wave's rows all see the keys [see_lo, see_hi)
    const int first = s.len - s.n + r0 / p.group;
    const int last = s.len - s.n + min(r0 + 32 * T::RT - 1, rows - 1) / p.group;
    const int see_hi = p.causal ? min(first + 1, s.len) : s.len;
    const int see_lo = p.window ? last - p.window + 1 : 0;

    const int32_t* table = p.table + static_cast<int64_t>(b) * p.width;
    const C* kb = static_cast<const C*>(p.k_cache) + h * p.head_stride;
    const C* vb = static_cast<const C*>(p.v_cache) + h * p.head_stride;
    char* const base = lds + wn * T::WAVE_BYTES;

    AttnStage<T> stage;
    int64_t off;
    uint64_t live;
    int t = ta + wn;
    if (t < tb) {
      look_up(p, table, t * T::KT, lo, hi, lane, off, live);
      load(kb, vb, off, live, st_id, stage);
      if (t + T::WN < tb) look_up(p, table, (t + T::WN) * T::KT, lo, hi, lane, off, live);
    }
    int buf = 0;
    for (; t < tb; t += T::WN) {
      char* lk = base + buf * 2 * T::TILE_BYTES;
      char* lv = lk + T::TILE_BYTES;
      store(lk, lv, st_id, stage);
      if (t + T::WN < tb) {
        load(kb, vb, off, live, st_id, stage);
        if (t + 2 * T::WN < tb) look_up(p, table, (t + 2 * T::WN) * T::KT, lo, hi, lane, off, live);
      }
      if constexpr (T::WM > 1) {
        // one barrier a tile: the buffer written next was last read before the barrier after that
        __syncthreads();
        buf ^= 1;
      } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      const int key0 = t * T::KT;
      const bool edge = key0 < see_lo || key0 + T::KT > see_hi;
      if (T::WM == 1 || r0 < rows)
        tile(lk, lv, key0, lane, edge, scale2, q, row_lo, row_hi, st);
      if constexpr (T::WM == 1) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
#pragma unroll
    for (int rt = 0; rt < T::RT; ++rt) st.l[rt] += __shfl_xor(st.l[rt], 32);

    if constexpr (T::WM > 1) {
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt) {
        const int rl = wm * 32 * T::RT + 32 * rt + (lane & 31);   // row in the tile
        const int r = m * T::BM + rl;
        if (r < rows) {
          if (slot >= 0 && lane < 32) g.part_ml[slot * T::BM + rl] = float2{st.m[rt], st.l[rt]};
#pragma unroll
          for (int i = 0; i < T::D / 32; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int d = 32 * i + 8 * x + 4 * (lane >> 5);
              const f32x4_t o = {st.o[rt][i][4 * x], st.o[rt][i][4 * x + 1], st.o[rt][i][4 * x + 2],
                                 st.o[rt][i][4 * x + 3]};
              if (slot >= 0)
                *reinterpret_cast<f32x4_t*>(g.part_o + (slot * T::BM + rl) * T::D + d) = o;
              else
                put(g, s, h, r, d, o, st.m[rt], st.l[rt], v_scale);
            }
        }
      }
      __syncthreads();   // the tiles in LDS are read: the next row tile may overwrite them
    } else {
      // join the waves' states through LDS, 32 rows at a time
      __shared__ float2 ml[T::WN][32];
#pragma unroll
      for (int rt = 0; rt < T::RT; ++rt) {
        const int qi = lane & 31;
#pragma unroll
        for (int i = 0; i < T::D / 32; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t c = 8 * i + 2 * x + (lane >> 5);   // 16-byte chunk of the row
            *reinterpret_cast<f32x4_t*>(base + qi * T::D * 4 + ((c ^ (qi & 15)) << 4)) =
                f32x4_t{st.o[rt][i][4 * x], st.o[rt][i][4 * x + 1], st.o[rt][i][4 * x + 2], st.o[rt][i][4 * x + 3]};
          }
        if (lane < 32) ml[wn][qi] = float2{st.m[rt], st.l[rt]};
        __syncthreads();
        for (int idx = static_cast<int>(threadIdx.x); idx < 32 * (T::D / 4); idx += T::THREADS) {
          const int qr = idx / (T::D / 4), c = idx % (T::D / 4);
          const int rl = 32 * rt + qr;
          const int r = m * T::BM + rl;
          if (r < rows) {
            float mm = ml[0][qr].x;
#pragma unroll
            for (int w = 1; w < T::WN; ++w) mm = fmaxf(mm, ml[w][qr].x);
            const float ref = mm == -INFINITY ? 0.f : mm;
            float l = 0.f;
            f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < T::WN; ++w) {
              const float f = __builtin_amdgcn_exp2f(ml[w][qr].x - ref);
              l += f * ml[w][qr].y;
              const f32x4_t ow =
                  *reinterpret_cast<const f32x4_t*>(lds + w * T::WAVE_BYTES + qr * T::D * 4 + ((c ^ (qr & 15)) << 4));
              o += f * ow;
            }
            if (slot >= 0) {
              *reinterpret_cast<f32x4_t*>(g.part_o + (slot * T::BM + rl) * T::D + 4 * c) = o;
              if (c == 0) g.part_ml[slot * T::BM + rl] = float2{mm, l};
            } else {
              put(g, s, h, r, 4 * c, o, mm, l, v_scale);
            }
          }
        }
        __syncthreads();
      }
    }
  }
};

// The workgroup's share of all key tiles, row tile by row tile.
template <typename T>
__global__ __launch_bounds__(T::THREADS) void attn_kernel(const AttnArgs g) {
  using Plan = AttnPlan<T::BM, T::KT>;
  __shared__ __attribute__((aligned(16))) char lds[T::LDS_BYTES];
  const AttnProblem& p = g.p;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  // neighbouring shares, which read the same keys, on one XCD
  const int64_t per_xcd = (g.slabs + 7) / 8;
  const int64_t w = static_cast<int64_t>(blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
  if (w >= g.slabs) return;   // whole workgroup
  // every wave sums and searches for itself: no barriers
  int64_t all = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    const int b = b0 + lane;
    all += b < p.batch ? Plan::total(p, Plan::seq(p, g.whole, b)) : 0;
  }
  all = uniform_i64(wave_sum_i64(all));
  const int64_t share = g.whole ? 1 : max(g.min_share, (all + g.slabs - 1) / g.slabs);
  int64_t x = w * share;
  const int64_t end = min(x + share, all);
  if (x >= end) {
    if (threadIdx.x == 0 && !g.whole) g.record[w * kRecord + 4] = -1;
    return;
  }
  // the request that holds x
  int b = 0;
  int64_t base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    const int bl = b0 + lane;
    int64_t c = bl < p.batch ? Plan::total(p, Plan::seq(p, g.whole, bl)) : 0;
    const int64_t own = c;
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
  int64_t in_req = x - base;
  int64_t unit = in_req / s.cost;
  int inner = static_cast<int>(in_req - unit * s.cost);
  int h = static_cast<int>(unit / s.units);
  int u = static_cast<int>(unit - static_cast<int64_t>(h) * s.units);
  bool fresh = true;   // nothing done yet: a partial here is continued from the workgroup before
  if (threadIdx.x == 0 && !g.whole) g.record[w * kRecord + 4] = -1;
  while (x < end) {
    // the unit's row tiles: the longer, then (paired) the shorter
    int done = 0;
    for (int part = 0; part < 2 && x < end; ++part) {
      int m;
      if (s.paired) {
        m = part == 0 ? s.tiles - 1 - u : u;
        if (part == 1 && m == s.tiles - 1 - u) break;
      } else {
        if (part == 1) break;
        m = u;
      }
      int lo, hi, t0, t1;
      Plan::range(p, s, m, lo, hi, t0, t1);
      const int nt = t1 - t0;
      if (g.whole) {
        AttnBody<T>::run(g, s, b, h, m, t0, t1, lo, hi, -1, lds);
        x += 1;
        fresh = false;
        break;
      }
      if (inner < done + nt) {
        const int from = inner - done;
        const int to = static_cast<int>(min(static_cast<int64_t>(nt), from + (end - x)));
        int64_t slot = -1;
        if (from > 0) {
          slot = 2 * w;
          if (threadIdx.x == 0 && fresh) {
            // x - from is where the row tile begins; the first border inside it does the join
            const int64_t x0 = x - from;
            int32_t* rec = g.record + w * kRecord;
            rec[0] = s.first;
            rec[1] = s.n;
            rec[2] = h;
            rec[3] = m;
            rec[4] = x0 / share == w - 1 ? static_cast<int32_t>((x0 + nt - 1) / share) : -1;
          }
        } else if (to < nt) {
          slot = 2 * w + 1;
        }
        AttnBody<T>::run(g, s, b, h, m, t0 + from, t0 + to, lo, hi, slot, lds);
        x += to - from;
        inner += to - from;
        fresh = false;
      }
      done += nt;
    }
    if (x >= end) break;
    if (!g.whole) x += s.cost - inner;   // what the unit costs less than its request's units at most
    inner = 0;
    if (++u == s.units) {
      u = 0;
      if (++h == p.hkv) {
        h = 0;
        do {
          if (++b >= p.batch) return;
          s = Plan::seq(p, g.whole, b);
        } while (s.units == 0);
      }
    }
  }
}

// Joins the partials of the row tiles that several workgroups share: blockIdx.x + 1 is
// the workgroup whose share begins inside one, blockIdx.y the rows.
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs g) {
  const AttnProblem& p = g.p;
  const int64_t w = blockIdx.x + 1;
  const int32_t* rec = g.record + w * kRecord;
  const int last = rec[4];
  if (last < 0) return;
  AttnSeq s{};
  s.first = rec[0];
  s.n = rec[1];
  const int h = rec[2], m = rec[3];
  float v_scale = 1.f;
  if constexpr (sizeof(typename T::C) == 1) v_scale = p.v_scale[h];
  constexpr int PER = 256 / (T::D / 4);   // rows at a time
  const int c = static_cast<int>(threadIdx.x) % (T::D / 4);
  for (int rl = blockIdx.y * PER + static_cast<int>(threadIdx.x) / (T::D / 4); rl < T::BM;
       rl += PER * static_cast<int>(gridDim.y)) {
    const int r = m * T::BM + rl;
    if (r >= s.n * p.group) break;
    float mm = -INFINITY;
    for (int64_t i = w - 1; i <= last; ++i)
      mm = fmaxf(mm, g.part_ml[(i == w - 1 ? 2 * i + 1 : 2 * i) * T::BM + rl].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float l = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int64_t i = w - 1; i <= last; ++i) {
      const int64_t slot = i == w - 1 ? 2 * i + 1 : 2 * i;
      const float2 ml = g.part_ml[slot * T::BM + rl];
      const float f = __builtin_amdgcn_exp2f(ml.x - ref);
      l += f * ml.y;
      o += f * *reinterpret_cast<const f32x4_t*>(g.part_o + (slot * T::BM + rl) * T::D + 4 * c);
    }
    AttnBody<T>::put(g, s, h, r, 4 * c, o, mm, l, v_scale);
  }
}

}  // namespace bdr
