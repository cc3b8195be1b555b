// Logits products of the vocabulary losses: softmax statistics and d logits.
//
// Few rows are bound by streaming the weight, which one row of tiles reads once:
// row tiles no taller than needed, as many stages as fit (128 x 320: three of the
// weight's and two of the hidden states', which come from L2), and non-temporal loads
// where the weight is larger than the last-level cache.  Many rows are bound by the
// matrix cores: the largest tile whose accumulators fit two waves per SIMD.  Where
// those tiles leave much of the chip idle (a small vocabulary), smaller ones.
// Measured (bf16, statistics):
//   H = 5120, V = 151936:
//     rows 7    64 x 320 227 us (6.8 TB/s; 257 us with temporal loads), 32 x 128 228 us,
//               128 x 320 234 us
//     rows 64   64 x 320 239 us, 128 x 320 242 us, 32 x 128 413 us
//     rows 128  128 x 320 257 us (two stages of both 295 us), 64 x 320 438 us
//     rows 256  256 x 320 383 us, 128 x 320 443 us
//     rows 4096, 20 x 2560 entries: 256 x 320 1577 us (1362 TFLOP/s; the library's
//               product of V entries 1326 - 1369), 256 x 256 with three and two
//               stages 1696 us, 128 x 320 1897 us, 128 x 128 2167 us
//   H = 5120, V = 64000, rows 100: 128 x 320 115 us (126 us temporal), 128 x 128 128 us
//   H = 2560, V = 26455, rows 128 (the weight stays in the last-level cache): 64 x 320
//               36 us (50 us non-temporal), 128 x 128 41 us, 128 x 320 48 us
//   H = 2552, V = 151936, rows 7: 64 x 320 160 us (203 us non-temporal: rows that are no
//               multiple of 128 bytes end inside a cache line, which the next step
//               then fetches again)
//   H = 1024, rows 64, V = 16384: 32 x 128 10 us, 128 x 128 17 us, 64 x 320 20 us

#include "loss.h"

namespace bdr {

namespace {

using LogitsF32 = LossTile<float, false, false, 2, 2, 2, 2, 2>;            // 64 x 64
using LogitsSmall = LossTile<uint16_t, false, false, 1, 4, 2, 2, 4>;       // 32 x 128
using LogitsMid = LossTile<uint16_t, false, false, 2, 2, 4, 4, 2>;         // 128 x 128
using LogitsFew = LossTile<uint16_t, false, false, 2, 4, 2, 5, 3>;         // 64 x 320
using LogitsSome = LossTile<uint16_t, false, false, 2, 4, 4, 5, 3, false, false, 2>;   // 128 x 320
using LogitsSomeOnce = LossTile<uint16_t, false, false, 2, 4, 4, 5, 3, false, true, 2>;
using LogitsMany = LossTile<uint16_t, false, false, 2, 4, 8, 5, 2>;        // 256 x 320

static_assert(kJoinRows == 64, "the rows of one FewRowsOnce tile");
// up to kJoinRows rows
using FewRowsSmall = LossTile<uint16_t, false, false, 1, 4, 2, 2, 4, false, false, 4, kJoinSteps>;
using FewRowsMid = LossTile<uint16_t, false, false, 2, 2, 4, 4, 2, false, false, 2, kJoinSteps>;
using FewRowsFew = LossTile<uint16_t, false, false, 2, 4, 2, 5, 3, false, false, 3, kJoinSteps>;
using FewRowsOnce = LossTile<uint16_t, false, false, 2, 4, 2, 5, 3, false, true, 3, kJoinSteps>;

// Microseconds of a product on tiles T: rounds of workgroups over the chip times its
// steps of 64 elements times `step` (of a full chip, from the times above), and no
// less than it takes to read a weight from HBM (6.6 TB/s non-temporal, else 5.2).
template <typename T>
double logits_us(int64_t rows, int64_t cols, int64_t hidden, double step, bool once) {
  const int64_t slots = 256 * T::PER_CU;
  const int64_t rounds = (loss_tiles<T>(rows, cols) + slots - 1) / slots;
  const double us = static_cast<double>(rounds * ((hidden + 63) / 64)) * step;
  if (!beyond_cache(cols * hidden)) return us;
  return std::max(us, static_cast<double>(cols * hidden * 2) / (once ? 6.6e6 : 5.2e6));
}

template <typename F>
auto with_logits_tile(bdr_dtype dt, int64_t rows, int64_t cols, int64_t hidden, F&& f) {
  if (dt != BDR_BF16) return f(LogitsF32{});
  const bool stream = beyond_cache(cols * hidden) && hidden % 64 == 0;
  const bool few_rows = rows <= kJoinRows;
  const bool few_once = stream && few_rows, some_once = stream && rows <= LogitsSome::BM;
  // (few rows are summed in blocks and have d logits of two terms, which the tall tiles do not)
  const double t[5] = {logits_us<LogitsFew>(rows, cols, hidden, 1.2, few_once),
                       few_rows ? 1e30 : logits_us<LogitsSome>(rows, cols, hidden, 1.3, some_once),
                       few_rows ? 1e30 : logits_us<LogitsMany>(rows, cols, hidden, 2.1, false),
                       logits_us<LogitsMid>(rows, cols, hidden, 1.15, false),
                       logits_us<LogitsSmall>(rows, cols, hidden, 0.85, false)};
  const int best = static_cast<int>(std::min_element(t, t + 5) - t);
  if (few_rows) {
    if (best == 0) return few_once ? f(FewRowsOnce{}) : f(FewRowsFew{});
    if (best == 3) return f(FewRowsMid{});
    return f(FewRowsSmall{});
  }
  if (best == 0) return f(LogitsFew{});
  if (best == 1) return some_once ? f(LogitsSomeOnce{}) : f(LogitsSome{});
  if (best == 2) return f(LogitsMany{});
  if (best == 3) return f(LogitsMid{});
  return f(LogitsSmall{});
}

}  // namespace

int loss_stats_cols(bdr_dtype dt, int64_t rows, int64_t cols, int64_t hidden) {
  return with_logits_tile(dt, rows, cols, hidden, [](auto t) { return decltype(t)::BN; });
}

hipError_t launch_loss_stats(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return with_logits_tile(dt, rows, g.N, g.seg[0].k, [&](auto t) {
    return launch_loss_gemm<decltype(t), LE_STATS>(g, stream);
  });
}

hipError_t launch_loss_dlogits(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream) {
  return with_logits_tile(dt, rows, g.N, g.seg[0].k, [&](auto t) {
    return launch_loss_gemm<decltype(t), LE_DLOGITS>(g, stream);
  });
}

}  // namespace bdr
