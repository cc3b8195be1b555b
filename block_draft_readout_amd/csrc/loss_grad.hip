// Gradient products of the vocabulary losses: d hidden = d logits W and
// d weight = d logits^T hidden (and the Markov head's, as narrow as its rank).
//
// Measured (bf16, H = 5120):
//   d hidden, 4096 rows, 30720 entries: 256 x 320 1042 - 1121 us (1237 - 1149 TFLOP/s),
//     256 x 256 with 4 splits 1203 us, 128 x 128 2059 us
//   d hidden, 128 rows, 151936 entries: 128 x 320 with 16 splits 321 us, 128 x 128
//     with 12 splits 337 us; 7 rows: 32 x 256, 3 stages 292 us
//   d weight, 4096 rows, 30720 entries: 256 x 320 1090 us (1183 TFLOP/s),
//     256 x 256 1163 us, 128 x 128 1664 us

#include "loss.h"

namespace bdr {

namespace {

using FeatF32 = LossTile<float, false, true, 2, 2, 4, 4, 2>;         // 128 x 128
using FeatNarrow = LossTile<uint16_t, false, true, 2, 2, 4, 2, 2>;   // 128 x 64
using FeatFew = LossTile<uint16_t, false, true, 1, 4, 2, 4, 3>;      // 32 x 256
using FeatSome = LossTile<uint16_t, false, true, 2, 4, 4, 5, 2>;     // 128 x 320
using FeatMany = LossTile<uint16_t, false, true, 2, 4, 8, 5, 2>;     // 256 x 320

using WeightF32 = LossTile<float, true, true, 2, 2, 4, 4, 2>;        // 128 x 128
using WeightNarrow = LossTile<uint16_t, true, true, 2, 2, 4, 2, 2>;  // 128 x 64
using WeightWide = LossTile<uint16_t, true, true, 2, 4, 8, 5, 2>;    // 256 x 320

constexpr int64_t kNarrowCols = 128;   // outputs this narrow take the narrow tiles

template <typename F>
auto with_feat_tile(bdr_dtype dt, int64_t rows, int64_t cols, F&& f) {
  if (dt != BDR_BF16) return f(FeatF32{});
  if (cols <= kNarrowCols) return f(FeatNarrow{});
  if (rows <= FeatFew::BM) return f(FeatFew{});
  if (rows <= FeatSome::BM) return f(FeatSome{});
  return f(FeatMany{});
}

}  // namespace

// As many reduction splits as fill the compute units once (a workgroup's LDS
// sets how many share one), each with at least 8 steps.
int loss_dfeat_splits(bdr_dtype dt, int64_t rows, int64_t cols, int64_t width) {
  return with_feat_tile(dt, rows, cols, [&](auto t) {
    using T = decltype(t);
    const int64_t tiles = (rows + T::BM - 1) / T::BM * ((cols + T::BN - 1) / T::BN);
    const int64_t slots = 256 * (160 * 1024 / T::LDS_BYTES);
    const int64_t steps = (width + T::KB - 1) / T::KB;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({slots / tiles, steps / 8, 64})));
  });
}

hipError_t launch_loss_dfeat(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return with_feat_tile(dt, rows, g.N, [&](auto t) {
    return launch_loss_gemm<decltype(t), LE_PARTIAL>(g, stream);
  });
}

hipError_t launch_loss_dweight(bdr_dtype dt, const LossGemm& g, hipStream_t stream) {
  if (dt != BDR_BF16) return launch_loss_gemm<WeightF32, LE_OUT>(g, stream);
  if (g.N <= kNarrowCols) return launch_loss_gemm<WeightNarrow, LE_OUT>(g, stream);
  return launch_loss_gemm<WeightWide, LE_OUT>(g, stream);
}

}  // namespace bdr
