// Logits products of the vocabulary losses: softmax statistics and d logits.
//
// Few rows are bound by streaming the weight: small row tiles, so that several
// loads of weight rows are in flight per compute unit; many rows by the matrix
// cores: the largest tile whose accumulators fit two waves per SIMD.  Measured
// (bf16, H = 5120, V = 151936; statistics):
//   rows 7:    32 x 128, 3 stages 260 us (6.0 TB/s); 32 x 256, 2 stages 332 us;
//              128 x 320 299 us
//   rows 128:  128 x 320 319 us; 128 x 128 406 us; 32 x 128 824 us
//   rows 4096 (30720 entries): 256 x 320 1010 us (1270 TFLOP/s; the library's
//              product 990 us in the same run); 256 x 256 and 128 x 128 9 % and
//              75 % slower

#include "loss.h"

namespace bdr {

namespace {

using LogitsF32 = LossTile<float, false, false, 2, 2, 2, 2, 2>;          // 64 x 64
using LogitsFew = LossTile<uint16_t, false, false, 1, 4, 2, 2, 3>;       // 32 x 128
using LogitsSome = LossTile<uint16_t, false, false, 2, 4, 4, 5, 2>;      // 128 x 320
using LogitsMany = LossTile<uint16_t, false, false, 2, 4, 8, 5, 2>;      // 256 x 320

template <int EPI>
hipError_t logits(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  if (dt != BDR_BF16) return launch_loss_gemm<LogitsF32, EPI>(g, stream);
  if (rows <= LogitsFew::BM) return launch_loss_gemm<LogitsFew, EPI>(g, stream);
  if (rows <= LogitsSome::BM) return launch_loss_gemm<LogitsSome, EPI>(g, stream);
  return launch_loss_gemm<LogitsMany, EPI>(g, stream);
}

}  // namespace

int loss_stats_cols(bdr_dtype dt, int64_t rows) {
  if (dt != BDR_BF16) return LogitsF32::BN;
  if (rows <= LogitsFew::BM) return LogitsFew::BN;
  return rows <= LogitsSome::BM ? LogitsSome::BN : LogitsMany::BN;
}

hipError_t launch_loss_stats(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return logits<LE_STATS>(dt, rows, g, stream);
}

hipError_t launch_loss_dlogits(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return logits<LE_DLOGITS>(dt, rows, g, stream);
}

}  // namespace bdr
