// Gradient products of the vocabulary losses: d hidden = d logits W and
// d weight = d logits^T hidden (and the Markov head's, as narrow as its rank).
//
// Measured (bf16, H = 5120; "library": its product of the same size, same run):
//   d hidden, 4096 rows, 12 x 2560 entries: 256 x 320 918 us (1404 TFLOP/s; library
//     1310 - 1460 us), 256 x 256 with 4 splits 1203 us, 128 x 128 2059 us
//   d hidden, 151936 entries: 7 rows 64 x 320 225 us (6.9 TB/s; 258 us with temporal
//     loads), 128 x 320 250 us; 64 rows 239 and 265 us; 128 rows 128 x 256 with three
//     stages 266 us, 128 x 320 260 us with three of the weight's and 286 us with two;
//     256 rows 256 x 320 376 us, 128 x 320 512 us
//   d hidden, H = 2560, 26455 entries (in the last-level cache), 128 rows: 128 x 256
//     34 us (39 us non-temporal); H = 1024, 32000 entries: 24 us, 128 x 320 26 us
//   d embedding, rank 64: 128 rows, 151936 entries, 256 splits 15 us, 32 splits
//     36 us; 4096 rows, 12 x 2560 entries, 16 splits 43 us, 64 splits 73 us
//   d weight, 20 x 2560 entries: 4096 rows 256 x 320 1718 us (1250 TFLOP/s), 128 x 320
//     2000 us; 2048 rows 902 and 1052 us; 30 x 2560 entries: 1280 rows 934 and 1010
//     us, 1000 rows 794 and 815 us, 768 rows 657 and 646 us, 512 rows 512 and 473 us
//     (H = 2560: 490 and 526, 420 and 435, 351 and 348, 268 and 255 us)
//   d weight, 151936 entries (1.56 GB written): 128 rows 128 x 320 376 us by itself and
//     444 us in a traced step, where one tile per workgroup takes 579 us; 7 rows 269 - 311 us
//   d w2, rank 64, 151936 entries: 4096 rows 231 us (5.4 TB/s of d logits; 2 stages
//     231 us), 1000 rows 62 us (2 stages 65 us), 128 rows 15.7 us (14.8 us)

#include "loss.h"

namespace bdr {

namespace {

using FeatF32 = LossTile<float, false, true, 2, 2, 2, 2, 2>;         // 64 x 64
using FeatNarrow = LossTile<uint16_t, false, true, 2, 2, 4, 2, 3>;   // 128 x 64
using FeatFew = LossTile<uint16_t, false, true, 2, 4, 2, 5, 3>;      // 64 x 320
using FeatFewOnce = LossTile<uint16_t, false, true, 2, 4, 2, 5, 3, false, true>;
using FeatSome = LossTile<uint16_t, false, true, 2, 4, 4, 4, 3>;     // 128 x 256
using FeatSomeOnce = LossTile<uint16_t, false, true, 2, 4, 4, 4, 3, false, true>;
using FeatMany = LossTile<uint16_t, false, true, 2, 4, 8, 5, 2>;     // 256 x 320

using WeightF32 = LossTile<float, true, true, 2, 2, 2, 2, 2>;        // 64 x 64
using WeightNarrow = LossTile<uint16_t, true, true, 2, 2, 4, 2, 3>;  // 128 x 64
// walks its tiles: with few rows the output's bytes bound it, and its stores
// overlap the next tile's loads
using WeightFew = LossTile<uint16_t, true, true, 2, 4, 4, 5, 2, true>;   // 128 x 320
using WeightMany = LossTile<uint16_t, true, true, 2, 4, 8, 5, 2>;        // 256 x 320

constexpr int64_t kNarrowCols = 128;   // outputs this narrow take the narrow tiles
constexpr int64_t kManyRows = 896;     // between the rows measured above

// `small`: a product of a few billion operations at most, where the launches
// count: narrow tiles, so that both gradients of a kind go into one launch.
template <typename F>
auto with_feat_tile(bdr_dtype dt, int64_t rows, bool small, int64_t cols, int64_t width, F&& f) {
  if (dt != BDR_BF16) return f(FeatF32{});
  if (small || cols <= kNarrowCols) return f(FeatNarrow{});
  // one row of tiles reads the weight once: non-temporal where no cache would keep it
  const bool once = beyond_cache(cols * width);
  if (rows <= FeatFew::BM) return once ? f(FeatFewOnce{}) : f(FeatFew{});
  if (rows <= FeatSome::BM) return once ? f(FeatSomeOnce{}) : f(FeatSome{});
  return f(FeatMany{});
}

template <typename F>
auto with_weight_tile(bdr_dtype dt, int64_t rows, bool small, const LossGemm& g, F&& f) {
  if (dt != BDR_BF16) return f(WeightF32{});
  // narrow outputs, and ones whose wide tiles would leave half the chip idle
  if (small || g.N <= kNarrowCols || loss_tiles<WeightFew>(g.M, g.N) < 128) return f(WeightNarrow{});
  if (rows < kManyRows) return f(WeightFew{});
  return f(WeightMany{});
}

}  // namespace

// As many reduction splits as fill the compute units once (a workgroup's LDS
// sets how many share one), each with at least 4 steps.
int loss_dfeat_splits(bdr_dtype dt, int64_t rows, bool small, int64_t cols, int64_t width) {
  return with_feat_tile(dt, rows, small, cols, width, [&](auto t) {
    using T = decltype(t);
    const int64_t tiles = loss_tiles<T>(rows, cols);
    const int64_t slots = 256 * T::PER_CU;
    const int64_t steps = (width + T::KB - 1) / T::KB;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({slots / tiles, steps / 4, 256})));
  });
}

hipError_t launch_loss_dfeat(bdr_dtype dt, int64_t rows, bool small, const LossGemm* x,
                             const LossGemm* e, hipStream_t stream) {
  if (x && e && dt != BDR_BF16) return launch_loss_gemm_pair<FeatF32, LE_PARTIAL>(*x, *e, stream);
  if (x && e && small) return launch_loss_gemm_pair<FeatNarrow, LE_PARTIAL>(*x, *e, stream);
  for (const LossGemm* g : {x, e}) {
    if (!g) continue;
    const hipError_t err = with_feat_tile(dt, rows, small, g->N, g->seg[0].k, [&](auto t) {
      return launch_loss_gemm<decltype(t), LE_PARTIAL>(*g, stream);
    });
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_loss_dweight(bdr_dtype dt, int64_t rows, bool small, const LossGemm* x,
                               const LossGemm* e, hipStream_t stream) {
  if (x && e && dt != BDR_BF16) return launch_loss_gemm_pair<WeightF32, LE_OUT>(*x, *e, stream);
  if (x && e && small) return launch_loss_gemm_pair<WeightNarrow, LE_OUT>(*x, *e, stream);
  for (const LossGemm* g : {x, e}) {
    if (!g) continue;
    const hipError_t err = with_weight_tile(dt, rows, small, *g, [&](auto t) {
      return launch_loss_gemm<decltype(t), LE_OUT>(*g, stream);
    });
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace bdr
