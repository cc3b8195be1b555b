// Logits products of the vocabulary losses: softmax statistics and d logits.
//
// Few rows are bound by streaming the weight, which one row of tiles reads once:
// row tiles no taller than needed, non-temporal loads, as many stages as fit.
// Many rows are bound by the matrix cores: the largest tile whose accumulators
// fit two waves per SIMD.  Where those tiles leave much of the chip idle (a small
// vocabulary), smaller ones.  Measured (bf16, statistics):
//   H = 5120, V = 151936:
//     rows 7    64 x 320 228 us (6.8 TB/s; 257 us with temporal loads),
//               32 x 128 229 us, 128 x 320 282 us
//     rows 64   64 x 320 239 us, 128 x 320 287 us, 32 x 128 479 us
//     rows 128  128 x 320 298 us (317 us temporal), 64 x 320 438 us
//     rows 256  256 x 320 395 us, 128 x 320 552 us (non-temporal 598 us), 64 x 320
//               952 us, 32 x 128 1795 us
//     rows 4096, 12 x 2560 entries: 256 x 320 1010 us (1270 TFLOP/s; the library's
//               product 990 us in the same run), 256 x 256 and 128 x 128 9 % and
//               75 % slower
//   H = 1024, V = 16384, rows 64: 32 x 128 13.7 us, 64 x 320 20.1 us
//   H = 2552, V = 26455, rows 312: 128 x 320 71 us, 128 x 128 135 us

#include "loss.h"

namespace bdr {

namespace {

using LogitsF32 = LossTile<float, false, false, 2, 2, 2, 2, 2>;                       // 64 x 64
using LogitsSmall = LossTile<uint16_t, false, false, 1, 4, 2, 2, 4, false, true>;     // 32 x 128
using LogitsMid = LossTile<uint16_t, false, false, 2, 2, 4, 4, 2>;                    // 128 x 128
using LogitsFew = LossTile<uint16_t, false, false, 2, 4, 2, 5, 3, false, true>;       // 64 x 320
using LogitsSome = LossTile<uint16_t, false, false, 2, 4, 4, 5, 2>;                   // 128 x 320
using LogitsSomeOnce = LossTile<uint16_t, false, false, 2, 4, 4, 5, 2, false, true>;  // non-temporal
using LogitsMany = LossTile<uint16_t, false, false, 2, 4, 8, 5, 2>;                   // 256 x 320

// Time of a product in units of one reduction step: rounds of workgroups over
// the chip times a step of that tile (microseconds per 64 elements with the chip
// full, from the times above over their rounds and steps).
template <typename T>
double rounds(int64_t rows, int64_t cols, double step) {
  const int64_t slots = 256 * T::PER_CU;
  return static_cast<double>((loss_tiles<T>(rows, cols) + slots - 1) / slots) * step;
}

template <typename F>
auto with_logits_tile(bdr_dtype dt, int64_t rows, int64_t cols, F&& f) {
  if (dt != BDR_BF16) return f(LogitsF32{});
  const double t[5] = {rounds<LogitsMany>(rows, cols, 2.45), rounds<LogitsSome>(rows, cols, 1.72),
                       rounds<LogitsFew>(rows, cols, 1.45), rounds<LogitsMid>(rows, cols, 1.25),
                       rounds<LogitsSmall>(rows, cols, 1.18)};
  const int best = static_cast<int>(std::min_element(t, t + 5) - t);
  if (best == 0) return f(LogitsMany{});
  if (best == 1) return rows <= LogitsSome::BM ? f(LogitsSomeOnce{}) : f(LogitsSome{});
  if (best == 2) return f(LogitsFew{});
  if (best == 3) return f(LogitsMid{});
  return f(LogitsSmall{});
}

}  // namespace

int loss_stats_cols(bdr_dtype dt, int64_t rows, int64_t cols) {
  return with_logits_tile(dt, rows, cols, [](auto t) { return decltype(t)::BN; });
}

hipError_t launch_loss_stats(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return with_logits_tile(dt, rows, g.N, [&](auto t) {
    return launch_loss_gemm<decltype(t), LE_STATS>(g, stream);
  });
}

hipError_t launch_loss_dlogits(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return with_logits_tile(dt, rows, g.N, [&](auto t) {
    return launch_loss_gemm<decltype(t), LE_DLOGITS>(g, stream);
  });
}

}  // namespace bdr
