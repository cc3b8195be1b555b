// The vocabulary losses that train a drafter (gfx950): softmax cross entropy
// and distillation from a teacher's top logits, over the logits the drafter
// drafts with (LM head plus Markov bias), forward and backward, without the
// logits ever being stored.
//
//   z[n, v] = sum_h hidden[n, h] W[v, h] + sum_j w1[prev[n], j] w2[v, j]
//   lse[n]  = log sum_v exp(z[n, v] / T)
//   cross entropy (T = 1): loss = lse - z[label],    d z = g (softmax(z) - onehot)
//   distillation: t = softmax_j(u_j / T) over the row's valid entries,
//     loss = T^2 sum_j t_j (log t_j - z[id_j] / T + lse),
//     d z  = g T (softmax(z / T) - sum_j t_j onehot(id_j))
//
// The Markov embedding of the previous token is a second stretch of the
// reduction, so the logits are one product of [hidden | w1[prev]] with
// [W | w2], and the gradients are the two products of d z with these.
//
// Rows without a target take no part: a first pass compacts the others
// (hidden, embedding and per-row values) into the workspace, and every product
// runs on the compacted rows, whose count stays on the device.
//
// The forward pass keeps a maximum and a sum per row and vocabulary tile; the
// backward pass walks the vocabulary in pieces and recomputes a piece's logits
// straight into d z (the only logits-sized buffer, one piece wide).  Per-row
// values, softmax sums and d hidden across pieces are fp32; d z is rounded to
// the storage type, as an operand of matrix products has to be (for up to 64 rows
// of bf16 kept as two such terms; with more, what the label's entry loses is added to
// the gradients apart, to the weights' for up to 512 rows).
//
// Every sum has a fixed order: the same inputs give the same bits.

#include <algorithm>

#include "loss.h"

namespace bdr {

namespace {

constexpr int64_t kPieceBytes = int64_t(512) << 20;   // d logits of one piece, or
constexpr int64_t kPieceCols = 2560;                  // this many entries: pieces are multiples of it
constexpr int64_t kSmallProduct = int64_t(1) << 30;   // rows * hidden * vocab

constexpr int64_t kCountRows = 1024;                  // rows of a block of the compaction
constexpr int64_t kManyRows = 4096;                   // more take a count of the blocks first

// What the row kernels read and write, besides the products.
struct LossRows {
  const void* hidden;
  const void* w1;
  const void* w2;
  const void* w;
  const int32_t* prev;
  const int32_t* label;    // cross entropy: labels; distillation: 0 or -1 per row
  const int32_t* ids;      // distillation [rows, top]
  const void* u;
  int u_bf16;
  int64_t rows;
  int hidden_size, vocab, rank, top;
  float scale2, temperature;   // log2(e) / temperature
  const float* lse;        // backward inputs
  const float* loss_grad;
  // workspace
  int32_t* live;           // [1]
  int32_t* counts;         // [blocks of kCountRows rows] rows with a target, or NULL
  int32_t* pos;            // [rows] compacted row or -1
  int32_t* row_of;         // [live] original row
  int32_t* label_c;        // [live]
  int32_t* prev_c;         // [live] previous token or -1
  void* x;                 // [live, H]
  void* e;                 // [live, r]
  float* lse2;             // [live]
  float* lse_corr;         // [live] 2^-(what rounding lse2 left), fp32 tensors only
  float* coef;             // [live]
  float* resid;            // [live] what rounding d logits left at label_c, or NULL
  float* t;                // [rows, top]
  float2* stat;            // [live, tiles]
  int tiles;
  float* z_label;          // [live]
};

// ---------------------------------------------------------------- targets of the distillation
// t = softmax of a row's valid teacher logits over T, and whether it has any
// mass; one wave per row.  The maximum is taken off before the division: the
// difference of two close logits is exact, their quotients by a small T are not.
// `label` gets the row's heaviest entry, or -1.
__global__ __launch_bounds__(256) void distill_target_kernel(const LossRows g, int32_t* label) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (n >= g.rows) return;
  const int32_t* ids = g.ids + n * g.top;
  float v[BDR_MAX_TEACHER / 64];
  float mx = -INFINITY;
  bool any = false;
#pragma unroll
  for (int c = 0; c < BDR_MAX_TEACHER / 64; ++c) {
    const int j = c * 64 + lane;
    v[c] = -INFINITY;
    if (j < g.top && static_cast<uint32_t>(ids[j]) < static_cast<uint32_t>(g.vocab)) {
      v[c] = g.u_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(g.u)[n * g.top + j])
                      : static_cast<const float*>(g.u)[n * g.top + j];
    }
    mx = fmaxf(mx, v[c]);
    any |= !(v[c] == -INFINITY);
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) mx = fmaxf(mx, __shfl_xor(mx, m));
  const bool row_any = __ballot(any) != 0ull;
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < BDR_MAX_TEACHER / 64; ++c) {
    v[c] = v[c] == -INFINITY ? 0.f : expf((v[c] - mx) / g.temperature);
    sum += v[c];
  }
  sum = wave_sum(sum);
  float top_weight = 0.f;
#pragma unroll
  for (int c = 0; c < BDR_MAX_TEACHER / 64; ++c) top_weight = fmaxf(top_weight, v[c]);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) top_weight = fmaxf(top_weight, __shfl_xor(top_weight, m));
#pragma unroll
  for (int c = 0; c < BDR_MAX_TEACHER / 64; ++c) {
    const int j = c * 64 + lane;
    if (j < g.top) g.t[n * g.top + j] = row_any ? v[c] / sum : 0.f;
  }
  // the largest id among the entries of the largest weight (NaN weights: any listed id)
  int best = -1;
#pragma unroll
  for (int c = 0; c < BDR_MAX_TEACHER / 64; ++c) {
    const int j = c * 64 + lane;
    if (j < g.top && !(v[c] < top_weight) && static_cast<uint32_t>(ids[j]) < static_cast<uint32_t>(g.vocab))
      best = max(best, ids[j]);
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) best = max(best, __shfl_xor(best, m));
  if (lane == 0) label[n] = row_any ? best : -1;
}

// ---------------------------------------------------------------- compaction
// Rows with a target in each block of rows.
__global__ __launch_bounds__(256) void loss_count_kernel(const LossRows g) {
  __shared__ int counts[4];
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kCountRows;
  int c = 0;
  for (int64_t n = n0 + threadIdx.x; n < min(n0 + kCountRows, g.rows); n += 256)
    c += static_cast<uint32_t>(g.label[n]) < static_cast<uint32_t>(g.vocab);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) c += __shfl_xor(c, m);
  if ((threadIdx.x & 63) == 0) counts[threadIdx.x >> 6] = c;
  __syncthreads();
  if (threadIdx.x == 0) g.counts[blockIdx.x] = counts[0] + counts[1] + counts[2] + counts[3];
}

// One workgroup per row: counts the rows with a target before it (its place),
// copies its hidden state and its Markov embedding there.  Reading the labels
// before the row again in every workgroup is cheaper than a scan in a launch of
// its own (4 bytes a row from L2 against 2 H bytes copied) up to some thousand
// rows; with more, a launch counts each block of rows first, and a workgroup reads
// the blocks' counts and the labels of its own block only (forward call, H = 64,
// 1000 entries: 65536 rows 619 -> 145 us, 16384 rows 70 -> 44 us, 8191 rows 36 -> 31
// us; 4096 rows take the 21 us of 2048 rows without it).
template <typename S, bool BACKWARD>
__global__ __launch_bounds__(256) void loss_gather_kernel(const LossRows g, u32x4_t* clear,
                                                          int64_t clear16) {
  __shared__ int counts[4];
  const int64_t n = blockIdx.x;
  if (BACKWARD && n >= g.rows) {   // workgroups past the rows clear d w1
    for (int64_t i = (n - g.rows) * 256 + threadIdx.x; i < clear16; i += (gridDim.x - g.rows) * 256)
      clear[i] = u32x4_t{0, 0, 0, 0};
    return;
  }
  const uint32_t V = static_cast<uint32_t>(g.vocab);
  int c = 0;
  int64_t first = 0;   // rows before it are in the counts
  if (g.counts) {
    first = n / kCountRows * kCountRows;
    for (int64_t i = threadIdx.x; i < n / kCountRows; i += 256) c += g.counts[i];
  }
  for (int64_t i = first + threadIdx.x; i < n; i += 256) c += static_cast<uint32_t>(g.label[i]) < V;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) c += __shfl_xor(c, m);
  if ((threadIdx.x & 63) == 0) counts[threadIdx.x >> 6] = c;
  __syncthreads();
  const int at = counts[0] + counts[1] + counts[2] + counts[3];
  const int32_t label = g.label[n];
  const bool in = static_cast<uint32_t>(label) < V;
  const int32_t p = g.rank ? g.prev[n] : -1;
  const bool has_prev = static_cast<uint32_t>(p) < V;
  if (threadIdx.x == 0) {
    g.pos[n] = in ? at : -1;
    if (n == g.rows - 1) *g.live = at + (in ? 1 : 0);
    if (in) {
      g.label_c[at] = label;
      g.row_of[at] = static_cast<int32_t>(n);
      if (g.rank) g.prev_c[at] = has_prev ? p : -1;
      if (BACKWARD) {
        // lse in units of log2: rounded to fp32, it would move every probability of the row by up
        // to 7e-7.  bf16 d logits have 2^-8; fp32's get the rounding back as a factor.
        const double l2 = static_cast<double>(g.lse[n]) * 1.4426950408889634;
        const float hi = static_cast<float>(l2);
        g.lse2[at] = hi;
        if (sizeof(S) == 4)
          g.lse_corr[at] = __builtin_amdgcn_exp2f(fabsf(hi) < INFINITY ? static_cast<float>(hi - l2) : 0.f);
        g.coef[at] = g.loss_grad[n] * g.temperature;
      }
    }
  }
  if (!in) return;
  const int chunks = g.hidden_size / Elem<S>::PER16;
  const u32x4_t* src = reinterpret_cast<const u32x4_t*>(static_cast<const S*>(g.hidden) +
                                                        n * g.hidden_size);
  u32x4_t* dst = reinterpret_cast<u32x4_t*>(static_cast<S*>(g.x) +
                                            static_cast<int64_t>(at) * g.hidden_size);
  for (int i = static_cast<int>(threadIdx.x); i < chunks; i += 256) dst[i] = src[i];
  const int rchunks = g.rank / Elem<S>::PER16;
  if (static_cast<int>(threadIdx.x) < rchunks) {
    u32x4_t v{0, 0, 0, 0};
    if (has_prev)
      v = reinterpret_cast<const u32x4_t*>(static_cast<const S*>(g.w1) +
                                           static_cast<int64_t>(p) * g.rank)[threadIdx.x];
    reinterpret_cast<u32x4_t*>(static_cast<S*>(g.e) + static_cast<int64_t>(at) * g.rank)[threadIdx.x] = v;
  }
}

// ---------------------------------------------------------------- loss values
// A softmax denominator: exp(lse) = 2^m s, s the row's sum of 2^(z scale2 - m), kept apart and in
// 64 bits until a result is rounded once.  A loss takes the label's logit from m first: logits that
// share a large offset (2^20: half a step of lse in fp32 is 0.06) leave it whole.
struct RowLse {
  double m, log_s;
  __device__ float lse() const { return static_cast<float>(m * kLn2d + log_s); }
  // lse - z / T
  __device__ double less(float z, float scale2) const {
    return (m - static_cast<double>(z) * scale2) * kLn2d + log_s;
  }
  static constexpr double kLn2d = 0.69314718055994530942;
};

// one compacted row's, in every lane of a wave
__device__ __forceinline__ RowLse row_lse(const float2* stat, int tiles, int lane) {
  float2 v{-INFINITY, 0.f};
  for (int i = lane; i < tiles; i += 64) v = merge_stat(v, stat[i]);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1)
    v = merge_stat(v, float2{__shfl_xor(v.x, m), __shfl_xor(v.y, m)});
  // (a join of two pairs is not the same bits from both sides: the first lane's counts)
  return RowLse{__shfl(v.x, 0), log(static_cast<double>(__shfl(v.y, 0)))};
}

// one wave per original row
__global__ __launch_bounds__(256) void ce_loss_kernel(const LossRows g, float* loss, float* lse) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (n >= g.rows) return;
  const int p = g.pos[n];
  float l = 0.f, out = 0.f;
  if (p >= 0) {
    const RowLse d = row_lse(g.stat + static_cast<int64_t>(p) * g.tiles, g.tiles, lane);
    l = d.lse();
    out = static_cast<float>(d.less(g.z_label[p], g.scale2));
  }
  if (lane == 0) {
    loss[n] = out;
    lse[n] = l;
  }
}

// logits at the teacher's entries: picked[n, j] = z[n, id_j], bit for bit those that the softmax is
// made of, so that what summing them lost cancels in lse - z (a dot product in another order left
// 5e-5 of a confident row's loss).  A matrix product's element is one chain of MFMAs along the
// reduction, whatever the tile: this one walks that chain with sixteen entries' weight rows as one
// operand and the row's hidden state, in all sixteen columns, as the other, in pieces of 64 bytes of
// every row, a batch of pieces on its way while another is multiplied (1 row of 5120, 20 entries: 12
// us, bound by latency; dot products by whole workgroups took 5, twelve waves handing the sums on
// take 10; 4096 rows of 5120, 64 entries: 440 us, 6 TB/s; the dot products took 480).
// Grid (rows, entries / 16), a wave each.
constexpr int kPickAhead = 8;     // pieces of a batch

// JOIN: steps of two pieces that are summed by themselves, as the product's tiles do
template <typename S, int JOIN>
__global__ __launch_bounds__(64) void distill_pick_kernel(const LossRows g, float* picked) {
  constexpr int PER = Elem<S>::PER16;
  const int lane = static_cast<int>(threadIdx.x);
  const int r16 = lane & 15, grp = lane >> 4;
  const int64_t n = blockIdx.x;
  const int j0 = static_cast<int>(blockIdx.y) * 16;
  const int p = g.pos[n];
  int id = p >= 0 && j0 + r16 < g.top ? g.ids[n * g.top + j0 + r16] : -1;
  if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(g.vocab)) id = -1;
  // pieces of the hidden state, then of the embedding; two are a step of the product, and the
  // embedding starts a step
  const int first = (g.hidden_size + 8 * PER - 1) / (8 * PER) * 2;
  const int pieces = __ballot(id >= 0) == 0ull ? 0 : first + (g.rank + 4 * PER - 1) / (4 * PER);
  const int64_t row = max(p, 0), entry = max(id, 0);
  const S* x = static_cast<const S*>(g.x) + row * g.hidden_size;
  const S* w = static_cast<const S*>(g.w) + entry * g.hidden_size;
  const S* e = static_cast<const S*>(g.e) + row * g.rank;
  const S* w2 = static_cast<const S*>(g.w2) + entry * g.rank;
  typedef u32x4_t Batch[kPickAhead];
  auto load = [&](int c0, Batch& a, Batch& b) {   // zeros past a stretch's end, and past the last piece
    if (c0 < pieces && (c0 + kPickAhead) * 4 * PER <= g.hidden_size) {
      // whole pieces (an entry that is not listed reads row 0 and is dropped)
      const S* xc = x + (c0 * 4 + grp) * PER;
      const S* wc = w + (c0 * 4 + grp) * PER;
#pragma unroll
      for (int q = 0; q < kPickAhead; ++q) {
        a[q] = load16(xc + q * 4 * PER);
        b[q] = load16(wc + q * 4 * PER);
      }
      return;
    }
#pragma unroll
    for (int q = 0; q < kPickAhead; ++q) {
      const bool second = c0 + q >= first;
      const int col = ((second ? c0 + q - first : c0 + q) * 4 + grp) * PER;
      const bool in = c0 + q < pieces && col < (second ? g.rank : g.hidden_size);
      a[q] = in ? load16((second ? e : x) + col) : u32x4_t{0, 0, 0, 0};
      b[q] = in && id >= 0 ? load16((second ? w2 : w) + col) : u32x4_t{0, 0, 0, 0};
    }
  };
  static_assert(kPickAhead % 2 == 0 && (JOIN == 0 || kPickAhead % (2 * JOIN) == 0), "whole blocks");
  f32x4_t acc{0.f, 0.f, 0.f, 0.f}, part;
  auto multiply = [&](const Batch& a, const Batch& b) {
#pragma unroll
    for (int q = 0; q < kPickAhead; ++q) {
      if constexpr (JOIN > 0) {
        if (q % (2 * JOIN) == 0) part = f32x4_t{0.f, 0.f, 0.f, 0.f};
        part = mma16(b[q], a[q], part, S());
        if (q % (2 * JOIN) == 2 * JOIN - 1) acc += part;
      } else {
        acc = mma16(b[q], a[q], acc, S());
      }
    }
  };
  Batch a0, b0, a1, b1;
  load(0, a0, b0);
  for (int c = 0; c < pieces; c += 2 * kPickAhead) {
    load(c + kPickAhead, a1, b1);
    multiply(a0, b0);
    load(c + 2 * kPickAhead, a0, b0);
    multiply(a1, b1);
  }
  // a lane holds entries 4 grp .. + 3 in every column
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int j = 4 * grp + c;
    const bool listed = __shfl(id, j) >= 0;
    if (r16 == 0 && j0 + j < g.top) picked[n * g.top + j0 + j] = listed ? acc[c] : 0.f;
  }
}

// one wave per original row; entries without mass add nothing
__global__ __launch_bounds__(256) void distill_loss_kernel(const LossRows g, const float* picked,
                                                           float* loss, float* lse) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (n >= g.rows) return;
  const int p = g.pos[n];
  float l = 0.f, out = 0.f;
  if (p >= 0) {
    const RowLse d = row_lse(g.stat + static_cast<int64_t>(p) * g.tiles, g.tiles, lane);
    l = d.lse();
    for (int j = lane; j < g.top; j += 64) {
      const float t = g.t[n * g.top + j];
      if (t != 0.f) out += t * (logf(t) + static_cast<float>(d.less(picked[n * g.top + j], g.scale2)));
    }
    out = wave_sum(out) * (g.temperature * g.temperature);
  }
  if (lane == 0) {
    loss[n] = out;
    lse[n] = l;
  }
}

// ---------------------------------------------------------------- d logits at the teacher's entries
// The product wrote coef * softmax everywhere; the entries with teacher mass
// are written again from the stored logit, coef (softmax - sum of the row's t
// at this id).  An id listed twice is written twice with the same value.
template <typename S>
__global__ __launch_bounds__(256) void distill_fix_kernel(const LossRows g, const float* picked,
                                                          S* dz, int64_t panel, int v0, int width,
                                                          float scale2, int two) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int p = static_cast<int>(i / g.top);
  if (p >= *g.live) return;
  const int j = static_cast<int>(i - static_cast<int64_t>(p) * g.top);
  const int64_t n = g.row_of[p];
  const int32_t* ids = g.ids + n * g.top;
  const int id = ids[j];
  if (id < v0 || id >= v0 + width) return;
  float t = 0.f;
  for (int q = 0; q < g.top; ++q)
    if (ids[q] == id) t += g.t[n * g.top + q];
  float pr = __builtin_amdgcn_exp2f(__builtin_fmaf(picked[n * g.top + j], scale2, -g.lse2[p]));
  if constexpr (sizeof(S) == 4) pr *= g.lse_corr[p];
  const float v = g.coef[p] * (pr - t);
  constexpr int KB = 128 / static_cast<int>(sizeof(S));   // d logits lie in panels of KB columns
  S* at = dz + (id - v0) / KB * panel + (static_cast<int64_t>(p) << two) * KB + (id - v0) % KB;
  *at = rounded<S>(v);
  if constexpr (sizeof(S) == 2) {
    if (two) at[KB] = rounded<S>(left_over(v));
    if (g.resid && id == g.label_c[p]) g.resid[p] = left_over(v);
  }
}

// ---------------------------------------------------------------- gradients out
// The reduction splits (and terms) of the feature gradients added in order, and what
// rounding d logits left at the label: d hidden rounded and back at the original rows
// (zeros for rows without a target), d embedding fp32 at the compacted rows.  SL lanes
// share the splits of four columns and join through LDS: few rows have many splits and
// few columns to spread over the chip.
// Grid (rows, column blocks of d hidden, then of d embedding), 1024 / SL columns
// in a block.
template <typename S>
struct JoinArgs {
  const int32_t* live;
  const int32_t* pos;
  const float* part_x;
  const float* part_e;
  int splits_x, splits_e, hidden, rank, blocks_x, two;
  int64_t rows;
  S* dx;
  float* de;
  const float* resid;      // [live] d logits' rounding at label, or NULL
  const int32_t* label;    // [live]
  const S* w;              // [V, hidden]
  const S* w2;             // [V, rank]
};

template <typename S, int SL>
__global__ __launch_bounds__(256) void loss_join_kernel(const JoinArgs<S> g) {
  constexpr int QUADS = 256 / SL;
  __shared__ f32x4_t sums[SL > 1 ? 256 : 1];
  const int64_t n = blockIdx.x;
  const bool emb = static_cast<int>(blockIdx.y) >= g.blocks_x;   // uniform
  if (emb && n >= *g.live) return;
  const int p = emb ? static_cast<int>(n) : g.pos[n];
  const int q = static_cast<int>(threadIdx.x) % QUADS;
  const int sl = static_cast<int>(threadIdx.x) / QUADS;
  const int cols = emb ? g.rank : g.hidden;
  const int parts = (emb ? g.splits_e : g.splits_x) << g.two;   // splits, the terms of each
  const int c = ((static_cast<int>(blockIdx.y) - (emb ? g.blocks_x : 0)) * QUADS + q) * 4;
  f32x4_t v{0.f, 0.f, 0.f, 0.f};
  if (p >= 0 && c < cols) {
    const float* src = (emb ? g.part_e : g.part_x) + (static_cast<int64_t>(p) << g.two) * cols + c;
    const int64_t slab = (g.rows << g.two) * cols;
#pragma unroll 4
    for (int s = sl; s < parts; s += SL)
      v += *reinterpret_cast<const f32x4_t*>(src + (s >> g.two) * slab + (s & g.two) * cols);
  }
  if constexpr (SL > 1) {
    sums[threadIdx.x] = v;
    __syncthreads();
    if (sl > 0) return;
#pragma unroll
    for (int k = 1; k < SL; ++k) v += sums[k * QUADS + q];
  }
  if (c >= cols) return;
  if (g.resid && p >= 0)
    v += g.resid[p] * load4((emb ? g.w2 : g.w) + static_cast<int64_t>(g.label[p]) * cols + c);
  if (emb)
    store4(g.de + n * cols + c, v);
  else
    store4(g.dx + n * cols + c, v);
}

// d w1[prev] = sum of the embedding gradients of the rows with that previous
// token, in row order.  One workgroup per compacted row; the first row with a
// token does the sum for it (d w1 was cleared with the compaction).  A row looks
// back for an earlier one, a first row at all after it: rows times distinct
// tokens at most, and rows * V is limited (all tokens distinct, H = 64, V = 131072:
// with the product before it 0.24 of 1.5 ms for 4096 rows, 14 of 166 ms for 131072).
template <typename S>
__global__ __launch_bounds__(256) void loss_dw1_kernel(const LossRows g, const float* de, S* out) {
  __shared__ int list[256];
  __shared__ int wave_n[4];
  __shared__ float sums[256];
  const int live = *g.live;
  const int p = static_cast<int>(blockIdx.x);
  if (p >= live) return;
  const int tok = g.prev_c[p];
  if (tok < 0) return;
  const int tid = static_cast<int>(threadIdx.x);
  for (int base = 0; base < p; base += 2048) {   // most rows of a common token end here early
    int seen = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = base + k * 256 + tid;
      if (i < p) seen |= g.prev_c[i] == tok;
    }
    if (__syncthreads_or(seen)) return;
  }
  // column r of group gr of the workgroup: rows of the list strided by groups
  const int r = g.rank;
  const int groups = 256 / r;
  const int col = tid % r, gr = tid / r;
  const int lane = tid & 63, wave = tid >> 6;
  float acc = 0.f;
  for (int base = p; base < live; base += 256) {
    const int i = base + tid;
    const bool hit = i < live && g.prev_c[i] == tok;
    const unsigned long long b = __ballot(hit);
    if (lane == 0) wave_n[wave] = __popcll(b);
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) before += wave_n[w];
      total += wave_n[w];
    }
    if (hit) list[before + __popcll(b & ((1ull << lane) - 1ull))] = i;
    __syncthreads();
    if (gr < groups)
#pragma unroll 4
      for (int q = gr; q < total; q += groups) acc += de[static_cast<int64_t>(list[q]) * r + col];
    __syncthreads();   // the list is rewritten
  }
  sums[tid] = acc;
  __syncthreads();
  if (gr == 0) {
    float v = 0.f;
    for (int q = 0; q < groups; ++q) v += sums[q * r + col];
    out[static_cast<int64_t>(tok) * r + col] = rounded<S>(v);
  }
}

__global__ __launch_bounds__(256) void clear_kernel(u32x4_t* p, int64_t n16) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n16;
       i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = u32x4_t{0, 0, 0, 0};
}

// ---------------------------------------------------------------- plan and workspace
struct LossPlan {
  int64_t piece;       // vocabulary entries per piece (backward)
  int64_t ld;          // row length of the piece's d logits buffer
  int two;             // d logits in two terms (stored rows = rows << two)
  bool resid;          // what their rounding leaves at the label is added
  bool small;          // narrow tiles, fewer launches
  int splits_x, splits_e;
  int stat_tiles;
};

LossPlan plan_loss(const LossProblem& p) {
  LossPlan q{};
  const int64_t es = p.dt == BDR_BF16 ? 2 : 4;
  const int cols = loss_stats_cols(p.dt, p.rows, p.vocab, p.hidden);
  q.stat_tiles = static_cast<int>((p.vocab + cols - 1) / cols);
  // whole vocabulary where its d logits fit, else equal pieces
  q.two = p.dt == BDR_BF16 && p.rows <= kTwoTermRows;
  q.resid = p.dt == BDR_BF16 && !q.two;
  const int64_t rows = p.rows << q.two;
  int64_t most = kPieceBytes / (rows * es) / kPieceCols * kPieceCols;
  most = std::max<int64_t>(most, kPieceCols);
  const int64_t pieces = (p.vocab + most - 1) / most;
  q.piece = ((p.vocab + pieces - 1) / pieces + kPieceCols - 1) / kPieceCols * kPieceCols;
  q.piece = std::min(q.piece, p.vocab);
  q.ld = (q.piece + 63) / 64 * 64;
  q.small = p.rows * p.hidden <= kSmallProduct / p.vocab;
  q.splits_x = loss_dfeat_splits(p.dt, rows, q.small, p.hidden, q.piece);
  q.splits_e = p.rank ? loss_dfeat_splits(p.dt, rows, q.small, p.rank, q.piece) : 0;
  return q;
}

// Workspace layout; with base NULL only the size counts.
struct LossSpace {
  char* base;
  size_t used = 0;
  template <typename U> U* take(int64_t count) {
    U* p = reinterpret_cast<U*>(base + used);
    used += align256(static_cast<size_t>(count) * sizeof(U));
    return p;
  }
};

struct LossBuffers {
  LossRows r;
  int32_t* has;
  char* dz;
  float* part_x;
  float* part_e;
  float* de;               // [live, r]
};

size_t lay_out(const LossProblem& p, const LossPlan& q, bool backward, char* base, LossBuffers& b) {
  LossSpace s{base};
  const int64_t es = p.dt == BDR_BF16 ? 2 : 4;
  LossRows& r = b.r;
  r.live = s.take<int32_t>(1);
  r.counts = s.take<int32_t>(p.rows > kManyRows ? (p.rows + kCountRows - 1) / kCountRows : 0);
  if (p.rows <= kManyRows) r.counts = nullptr;
  r.pos = s.take<int32_t>(p.rows);
  r.row_of = s.take<int32_t>(p.rows);
  r.label_c = s.take<int32_t>(p.rows);
  r.prev_c = s.take<int32_t>(p.rows);
  r.x = s.take<char>(p.rows * p.hidden * es);
  r.e = s.take<char>(p.rows * p.rank * es);
  if (p.top) {
    r.t = s.take<float>(p.rows * p.top);
    b.has = s.take<int32_t>(p.rows);
  }
  if (!backward) {
    r.z_label = s.take<float>(p.rows);
    r.stat = s.take<float2>(p.rows * q.stat_tiles);
  } else {
    r.lse2 = s.take<float>(p.rows);
    r.lse_corr = s.take<float>(p.dt == BDR_F32 ? p.rows : 0);
    r.coef = s.take<float>(p.rows);
    const int64_t rows = p.rows << q.two;
    b.dz = s.take<char>(rows * q.ld * es);
    b.part_x = s.take<float>(q.splits_x * rows * p.hidden);
    b.part_e = s.take<float>(q.splits_e * rows * p.rank);
    b.de = s.take<float>(q.splits_e > 1 || q.two || q.resid ? p.rows * p.rank : 0);
    r.resid = s.take<float>(q.resid ? p.rows : 0);
    if (!q.resid) r.resid = nullptr;
  }
  return s.used;
}

void fill_rows(const LossProblem& p, const LossPlan& q, LossBuffers& b) {
  LossRows& r = b.r;
  r.hidden = p.x;
  r.w = p.w;
  r.w1 = p.w1;
  r.w2 = p.w2;
  r.prev = p.prev;
  r.label = p.top ? b.has : p.labels;
  r.ids = p.ids;
  r.u = p.u;
  r.u_bf16 = p.u_dt == BDR_BF16;
  r.rows = p.rows;
  r.hidden_size = static_cast<int>(p.hidden);
  r.vocab = static_cast<int>(p.vocab);
  r.rank = p.rank;
  r.top = p.top;
  r.temperature = p.temperature;
  r.scale2 = kLog2e / p.temperature;   // as the products' epilogues take it
  r.tiles = q.stat_tiles;
}

#define BDR_LAUNCH(x)                 \
  do {                                \
    const hipError_t e_ = (x);        \
    if (e_ != hipSuccess) return e_;  \
  } while (0)

unsigned waves4(int64_t rows) { return static_cast<unsigned>((rows + 3) / 4); }

template <typename S>
hipError_t gather(const LossProblem& p, const LossBuffers& b, bool backward, void* dw1,
                  hipStream_t st) {
  if (p.top) {
    hipLaunchKernelGGL(distill_target_kernel, dim3(waves4(p.rows)), dim3(256), 0, st, b.r, b.has);
    BDR_LAUNCH(hipGetLastError());
  }
  if (b.r.counts) {
    hipLaunchKernelGGL(loss_count_kernel,
                       dim3(static_cast<unsigned>((p.rows + kCountRows - 1) / kCountRows)), dim3(256),
                       0, st, b.r);
    BDR_LAUNCH(hipGetLastError());
  }
  if (backward) {
    const int64_t n16 = dw1 ? p.vocab * p.rank * static_cast<int64_t>(sizeof(S)) / 16 : 0;
    const int64_t blocks = p.rows + std::min<int64_t>((n16 + 255) / 256, 2048);
    hipLaunchKernelGGL((loss_gather_kernel<S, true>), dim3(static_cast<unsigned>(blocks)), dim3(256),
                       0, st, b.r, static_cast<u32x4_t*>(dw1), n16);
  } else {
    hipLaunchKernelGGL((loss_gather_kernel<S, false>), dim3(static_cast<unsigned>(p.rows)),
                       dim3(256), 0, st, b.r, nullptr, 0);
  }
  return hipGetLastError();
}

// the logits product over vocabulary entries [v0, v0 + width)
LossGemm logits_gemm(const LossProblem& p, const LossRows& r, int64_t v0, int64_t width) {
  const int64_t es = p.dt == BDR_BF16 ? 2 : 4;
  LossGemm g{};
  g.seg[0] = LossSeg{r.x, static_cast<const char*>(p.w) + v0 * p.hidden * es, p.hidden, p.hidden,
                     p.hidden};
  if (p.rank)
    g.seg[1] = LossSeg{r.e, static_cast<const char*>(p.w2) + v0 * p.rank * es, p.rank, p.rank,
                       p.rank};
  else
    g.seg[1] = LossSeg{g.seg[0].a, g.seg[0].b, p.hidden, p.hidden, 0};
  g.live = r.live;
  g.M = p.rows;
  g.N = width;
  g.live_m = 1;
  g.band = 16;
  g.splits = 1;
  g.scale2 = kLog2e / p.temperature;
  return g;
}

template <typename S>
hipError_t forward(const LossProblem& p, void* workspace, float* loss, float* lse, float* picked,
                   hipStream_t st) {
  const LossPlan q = plan_loss(p);
  LossBuffers b{};
  lay_out(p, q, false, static_cast<char*>(workspace), b);
  fill_rows(p, q, b);
  BDR_LAUNCH(gather<S>(p, b, false, nullptr, st));
  LossGemm g = logits_gemm(p, b.r, 0, p.vocab);
  g.label = p.top ? nullptr : b.r.label_c;
  g.picked = b.r.z_label;
  g.stat = b.r.stat;
  BDR_LAUNCH(launch_loss_stats(p.dt, p.rows, g, st));
  if (p.top) {
    auto pick = [&](auto join) {
      hipLaunchKernelGGL((distill_pick_kernel<S, decltype(join)::value>),
                         dim3(static_cast<unsigned>(p.rows), static_cast<unsigned>((p.top + 15) / 16)),
                         dim3(64), 0, st, b.r, picked);
      return hipGetLastError();
    };
    if constexpr (sizeof(S) == 4)
      BDR_LAUNCH(pick(std::integral_constant<int, 1>{}));
    else
      BDR_LAUNCH(p.rows <= kJoinRows ? pick(std::integral_constant<int, kJoinSteps>{})
                                     : pick(std::integral_constant<int, 0>{}));
    hipLaunchKernelGGL(distill_loss_kernel, dim3(waves4(p.rows)), dim3(256), 0, st, b.r, picked,
                       loss, lse);
  } else {
    hipLaunchKernelGGL(ce_loss_kernel, dim3(waves4(p.rows)), dim3(256), 0, st, b.r, loss, lse);
  }
  return hipGetLastError();
}

// Many splits with 16 lanes each on four columns, few with one (128 rows of 5120,
// 16 splits: 54 us with one lane, 20 us with 16).
template <typename S>
hipError_t join(JoinArgs<S> g, hipStream_t st) {
  auto run = [&](auto lanes) {
    constexpr int SL = decltype(lanes)::value;
    constexpr int COLS = 1024 / SL;
    g.blocks_x = g.dx ? (g.hidden + COLS - 1) / COLS : 0;
    const int blocks_e = g.de ? (g.rank + COLS - 1) / COLS : 0;
    hipLaunchKernelGGL((loss_join_kernel<S, SL>),
                       dim3(static_cast<unsigned>(g.rows), static_cast<unsigned>(g.blocks_x + blocks_e)),
                       dim3(256), 0, st, g);
    return hipGetLastError();
  };
  if (g.dx ? g.splits_x >= 8 : g.splits_e >= 8)
    return run(std::integral_constant<int, 16>{});
  return run(std::integral_constant<int, 1>{});
}

template <typename S>
hipError_t backward(const LossProblem& p, const LossGrads& o, void* workspace, const float* lse,
                    const float* picked, const float* loss_grad, hipStream_t st) {
  const LossPlan q = plan_loss(p);
  const int64_t es = sizeof(S);
  const int64_t rows = p.rows << q.two;   // of d logits as stored
  LossBuffers b{};
  lay_out(p, q, true, static_cast<char*>(workspace), b);
  fill_rows(p, q, b);
  b.r.lse = lse;
  b.r.loss_grad = loss_grad;
  BDR_LAUNCH(gather<S>(p, b, true, o.w1, st));
  for (int64_t v0 = 0; v0 < p.vocab; v0 += q.piece) {
    const int64_t width = std::min(q.piece, p.vocab - v0);
    const int64_t ld = (width + 63) / 64 * 64;
    const int64_t panel = rows * (128 / es);   // elements of 128-byte columns
    LossGemm g = logits_gemm(p, b.r, v0, width);
    if (!p.top) {
      g.label = b.r.label_c;
      g.label0 = static_cast<int>(v0);
    }
    g.lse2 = b.r.lse2;
    g.lse_corr = b.r.lse_corr;
    g.coef = b.r.coef;
    g.out = b.dz;
    g.ldo = ld;
    g.slab = panel;
    g.two = q.two;
    g.resid = p.top ? nullptr : b.r.resid;   // (distillation: written with the teacher's entries)
    BDR_LAUNCH(launch_loss_dlogits(p.dt, p.rows, g, st));
    if (p.top) {
      hipLaunchKernelGGL(distill_fix_kernel<S>,
                         dim3(static_cast<unsigned>((p.rows * p.top + 255) / 256)), dim3(256), 0, st,
                         b.r, picked, reinterpret_cast<S*>(b.dz), panel, static_cast<int>(v0),
                         static_cast<int>(width), g.scale2, q.two);
      BDR_LAUNCH(hipGetLastError());
    }
    // d hidden and d embedding: reduction over this piece's entries
    auto dfeat = [&](const void* w, int64_t cols, float* part, int splits) {
      LossGemm d{};
      d.seg[0] = LossSeg{b.dz, static_cast<const char*>(w) + v0 * cols * es, panel, cols, width};
      d.seg[1] = LossSeg{d.seg[0].a, d.seg[0].b, panel, cols, 0};
      d.live = b.r.live;
      d.M = rows;
      d.N = cols;
      d.live_m = 1;
      d.band = 16;
      d.splits = splits;
      d.two = q.two;
      d.out = part;
      d.ldo = cols;
      d.slab = rows * cols;
      d.accumulate = v0 > 0;
      return d;
    };
    // d weight and d w2: reduction over the rows
    auto dweight = [&](const void* feat, int64_t cols, void* out) {
      LossGemm d{};
      d.seg[0] = LossSeg{b.dz, feat, panel, cols, rows};
      d.seg[1] = LossSeg{d.seg[0].a, d.seg[0].b, panel, cols, 0};
      d.live = b.r.live;
      d.M = width;
      d.N = cols;
      d.live_k = 1;
      d.two = q.two;
      d.label = b.r.label_c;
      d.label0 = static_cast<int>(v0);
      d.resid = p.rows <= kHeldRows ? b.r.resid : nullptr;
      // many rows: taller bands push the step's d logits out of an XCD's L2 (256 x 320
      // tiles, 4096 rows: 4 rows of tiles a band 1718 us, 16 1887 us; 1000 rows: 849 and
      // 798 us; 128 x 320 tiles, 768 rows: 16 646 us, 24 669 us; 128 rows in a traced step:
      // 4 519 us, 16 456 us, 24 444 us)
      d.band = p.rows <= 512 ? 24 : p.rows < 1536 ? 16 : 4;
      d.splits = 1;
      d.out = static_cast<char*>(out) + v0 * cols * es;
      d.ldo = cols;
      return d;
    };
    LossGemm gx, ge;
    if (o.hidden) gx = dfeat(p.w, p.hidden, b.part_x, q.splits_x);
    if (o.w1) ge = dfeat(p.w2, p.rank, b.part_e, q.splits_e);
    BDR_LAUNCH(launch_loss_dfeat(p.dt, rows, q.small, o.hidden ? &gx : nullptr,
                                 o.w1 ? &ge : nullptr, st));
    if (o.w) gx = dweight(b.r.x, p.hidden, o.w);
    if (o.w2) ge = dweight(b.r.e, p.rank, o.w2);
    BDR_LAUNCH(launch_loss_dweight(p.dt, rows, q.small, o.w ? &gx : nullptr,
                                   o.w2 ? &ge : nullptr, st));
  }
  const bool join_e = o.w1 && (q.splits_e > 1 || q.two || q.resid);
  if (o.hidden || join_e)
    BDR_LAUNCH(join(JoinArgs<S>{b.r.live, b.r.pos, b.part_x, b.part_e, q.splits_x, q.splits_e,
                                static_cast<int>(p.hidden), p.rank, 0, q.two, p.rows,
                                static_cast<S*>(o.hidden), join_e ? b.de : nullptr, b.r.resid,
                                b.r.label_c, static_cast<const S*>(p.w), static_cast<const S*>(p.w2)},
                    st));
  if (o.w1) {
    const float* de = join_e ? b.de : b.part_e;
    hipLaunchKernelGGL(loss_dw1_kernel<S>, dim3(static_cast<unsigned>(p.rows)), dim3(256), 0, st,
                       b.r, de, static_cast<S*>(o.w1));
    BDR_LAUNCH(hipGetLastError());
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_clear(void* p, int64_t bytes, hipStream_t stream) {
  const int64_t n16 = bytes / 16;
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((n16 + 255) / 256, 8192));
  hipLaunchKernelGGL(clear_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                     static_cast<u32x4_t*>(p), n16);
  return hipGetLastError();
}

size_t loss_workspace(const LossProblem& p, bool backward) {
  LossBuffers b{};
  return lay_out(p, plan_loss(p), backward, nullptr, b);
}

hipError_t launch_loss_forward(const LossProblem& p, void* workspace, float* loss, float* lse,
                               float* picked, hipStream_t stream) {
  return p.dt == BDR_BF16 ? forward<uint16_t>(p, workspace, loss, lse, picked, stream)
                          : forward<float>(p, workspace, loss, lse, picked, stream);
}

hipError_t launch_loss_backward(const LossProblem& p, const LossGrads& out, void* workspace,
                                const float* lse, const float* picked, const float* loss_grad,
                                hipStream_t stream) {
  return p.dt == BDR_BF16
             ? backward<uint16_t>(p, out, workspace, lse, picked, loss_grad, stream)
             : backward<float>(p, out, workspace, lse, picked, loss_grad, stream);
}

hipError_t launch_loss_clear(const LossProblem& p, const LossGrads& o, hipStream_t stream) {
  const int64_t es = p.dt == BDR_BF16 ? 2 : 4;
  if (o.w) BDR_LAUNCH(launch_clear(o.w, p.vocab * p.hidden * es, stream));
  if (o.w1) BDR_LAUNCH(launch_clear(o.w1, p.vocab * p.rank * es, stream));
  if (o.w2) BDR_LAUNCH(launch_clear(o.w2, p.vocab * p.rank * es, stream));
  return hipSuccess;
}

}  // namespace bdr
