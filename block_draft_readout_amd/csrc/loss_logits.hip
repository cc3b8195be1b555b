// Logits products of the vocabulary losses: softmax statistics and d logits.

#include "loss.h"

namespace bdr {

using LogitsF32 = LossTile<float, false, false, 2, 2, 4, 4, 2>;
using LogitsBf16 = LossTile<uint16_t, false, false, 2, 2, 4, 4, 2>;

int loss_stats_cols(bdr_dtype dt, int64_t rows) { return 128; }

hipError_t launch_loss_stats(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return dt == BDR_BF16 ? launch_loss_gemm<LogitsBf16, LE_STATS>(g, stream)
                        : launch_loss_gemm<LogitsF32, LE_STATS>(g, stream);
}

hipError_t launch_loss_dlogits(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return dt == BDR_BF16 ? launch_loss_gemm<LogitsBf16, LE_DLOGITS>(g, stream)
                        : launch_loss_gemm<LogitsF32, LE_DLOGITS>(g, stream);
}

}  // namespace bdr
