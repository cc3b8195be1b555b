// Gradient products of the vocabulary losses: d hidden = d logits W and
// d weight = d logits^T hidden.

#include "loss.h"

namespace bdr {

using FeatF32 = LossTile<float, false, true, 2, 2, 4, 4, 2>;
using FeatBf16 = LossTile<uint16_t, false, true, 2, 2, 4, 4, 2>;
using WeightF32 = LossTile<float, true, true, 2, 2, 4, 4, 2>;
using WeightBf16 = LossTile<uint16_t, true, true, 2, 2, 4, 4, 2>;

// Splits enough for two workgroups per compute unit, each with at least 8 steps.
int loss_dfeat_splits(bdr_dtype dt, int64_t rows, int64_t cols, int64_t width) {
  const int64_t tiles = (rows + 127) / 128 * ((cols + 127) / 128);
  const int64_t steps = (width * (dt == BDR_BF16 ? 2 : 4) + 127) / 128;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({512 / tiles, steps / 8, 64})));
}

hipError_t launch_loss_dfeat(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return dt == BDR_BF16 ? launch_loss_gemm<FeatBf16, LE_PARTIAL>(g, stream)
                        : launch_loss_gemm<FeatF32, LE_PARTIAL>(g, stream);
}

hipError_t launch_loss_dweight(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return dt == BDR_BF16 ? launch_loss_gemm<WeightBf16, LE_OUT>(g, stream)
                        : launch_loss_gemm<WeightF32, LE_OUT>(g, stream);
}

}  // namespace bdr
