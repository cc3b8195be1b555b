// Host-side description of one vocabulary-loss call (cross entropy or
// distillation), shared by the loss translation units.
#pragma once

#include "loss_gemm.h"

namespace bdr {

// Kinds of matrix products, each with its own translation unit:
// the logits' statistics and d logits (reduction fast on both sides), d hidden
// (d logits fast, weights slow) and d weight (both slow).
hipError_t launch_loss_stats(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream);
hipError_t launch_loss_dlogits(bdr_dtype dt, int64_t rows, const LossGemm& g, hipStream_t stream);
// the gradients of hidden and embedding, or of W and w2 (either may be NULL), in
// one launch where they take the same tiles
hipError_t launch_loss_dfeat(bdr_dtype dt, int64_t rows, bool small, const LossGemm* x,
                             const LossGemm* e, hipStream_t stream);
hipError_t launch_loss_dweight(bdr_dtype dt, int64_t rows, bool small, const LossGemm* x,
                               const LossGemm* e, hipStream_t stream);

// output tiles of tile shape T
template <typename T>
int64_t loss_tiles(int64_t rows, int64_t cols) {
  return (rows + T::BM - 1) / T::BM * ((cols + T::BN - 1) / T::BN);
}

// bf16 d logits of up to this many rows are kept as the sum of two bf16 terms, 16 bits:
// the products then have twice the rows, which costs little while the weight's bytes
// bound them (a step of 128 rows of 5120 would go from 1287 to 1581 us).  One term's
// rounding adds to a gradient about the error of its own rounding (1.4 times in all,
// relative to the norm); over a few dozen rows it scatters, 1.0 to 1.9 times.  More rows
// get back in fp32 what the rounding takes from the label's entry (at most 1.5 times over
// 78 drawn problems; a step of 128 rows of 5120 1283 -> 1307 us).
constexpr int64_t kTwoTermRows = 64;

// Logits of up to this many bf16 rows are summed in blocks of kJoinSteps steps (fp32's of one): the
// loss of a confident row is a small difference, and a few rows' errors do not average out (one row
// of 3528: 3.3e-6 of its loss as a chain of MFMAs, a vector product in fp32 5e-7).  Tiles for more
// rows have no registers for it.
constexpr int64_t kJoinRows = kTwoTermRows;
constexpr int kJoinSteps = 4;

// Weights larger than the last-level cache (256 MiB) stay in HBM between the products
// that read them: bytes of `n` bf16 entries above that.
inline bool beyond_cache(int64_t n) { return n * 2 > (int64_t(256) << 20); }

// vocabulary columns of one statistics tile
int loss_stats_cols(bdr_dtype dt, int64_t rows, int64_t cols, int64_t hidden);
// reduction splits of a d hidden product over `width` vocabulary entries
int loss_dfeat_splits(bdr_dtype dt, int64_t rows, bool small, int64_t cols, int64_t width);

}  // namespace bdr
