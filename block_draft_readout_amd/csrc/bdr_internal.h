// Host-side interface between the C ABI layer and the kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/bdr.h"
#include "gemm_plan.h"

namespace bdr {

// ----------------------------------------------------------------------------
// Markov bias + semi-autoregressive argmax over k positions.
// ----------------------------------------------------------------------------
size_t markov_workspace(int64_t B, int k);
hipError_t launch_markov(const float* logits, int64_t B, int k, int64_t V, bdr_dtype wdt,
                         const void* w1, const void* w2, int rank, const int32_t* prev,
                         int32_t* draft, int32_t* status, void* workspace, int n_cu,
                         hipStream_t stream);
// process-wide limit of the chain's bounded waits (negative / non-finite: default)
void set_poll_timeout_us(double us);
void set_forced_time_out(bool on);

// ----------------------------------------------------------------------------
// Greedy verification.
// ----------------------------------------------------------------------------
int verify_chunks(int64_t B, int k, int64_t V);
size_t verify_workspace(int64_t B, int k, int64_t V);
hipError_t launch_verify(const void* Y, bdr_dtype dt, int64_t B, int k, int64_t V,
                         const int32_t* draft, const float* conf, float threshold,
                         int32_t* block_len, int32_t* accepted, int32_t* bonus,
                         int32_t* target_argmax, int64_t* acc, int64_t* prop,
                         void* workspace, hipStream_t stream);

// ----------------------------------------------------------------------------
// Probabilistic drafting and rejection-sampling verification.
// ----------------------------------------------------------------------------
// noise[(b * k + i) * V + v] = Gumbel noise of stream stream_id at (b, i, v)
hipError_t launch_gumbel_noise(float* noise, int64_t B, int k, int64_t V, uint64_t seed,
                               uint32_t stream_id, hipStream_t stream);
size_t markov_sample_workspace(int64_t B, int k, int64_t V);
hipError_t launch_markov_sample(const float* logits, int64_t B, int k, int64_t V, bdr_dtype wdt,
                                const void* w1, const void* w2, int rank, const int32_t* prev,
                                float inv_t, uint64_t seed, int32_t* draft, float* xout,
                                const float* conf, float threshold, int32_t* status,
                                void* workspace, int n_cu, hipStream_t stream);
size_t sample_verify_workspace(int64_t B, int k, int64_t V);
hipError_t launch_verify_sample(const void* Y, bdr_dtype dt, int64_t B, int k, int64_t V,
                                const int32_t* draft, const float* X, const float* conf,
                                float threshold, float inv_t, uint64_t seed, int32_t* block_len,
                                int32_t* accepted, int32_t* bonus, int64_t* acc, int64_t* prop,
                                void* workspace, hipStream_t stream);

// ----------------------------------------------------------------------------
// Closing the loop: commit a verified block; the fc on gathered rows.
// ----------------------------------------------------------------------------
hipError_t launch_commit(const int32_t* draft, const int32_t* accepted, const int32_t* bonus,
                         const int32_t* block_len, int64_t B, int k, int32_t* next_prev,
                         int32_t* emitted, int32_t* draft_list, int32_t* row_index,
                         int32_t* row_count, int32_t* row_offsets, hipStream_t stream);
size_t fc_rows_workspace(int64_t max_rows, int64_t hidden, int n_taps, bdr_dtype dt);
hipError_t launch_fc_rows(const void* const* taps, int n_taps, int64_t rows, int64_t hidden,
                          bdr_dtype dt, const int32_t* row_index, const int32_t* row_count,
                          int64_t max_rows, const void* fc_w, void* out, void* workspace,
                          hipStream_t stream);
size_t fc_rows_fp8_workspace(int64_t max_rows, int64_t hidden, int n_taps);
hipError_t launch_fc_rows_fp8(const void* const* taps, int n_taps, int64_t rows, int64_t hidden,
                              const int32_t* row_index, const int32_t* row_count,
                              int64_t max_rows, const uint8_t* fc_q, const float* fc_scale,
                              void* out, void* workspace, hipStream_t stream);

// ----------------------------------------------------------------------------
// Row normalisation, forward and backward.
// ----------------------------------------------------------------------------
size_t norm_workspace(int64_t rows, int64_t hidden);
hipError_t launch_norm(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, bdr_dtype dt,
                       const void* w, const void* b, float eps, void* y, float* mean, float* rstd,
                       hipStream_t stream);
hipError_t launch_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                int64_t rows, int64_t hidden, bdr_dtype dt, const void* w,
                                const float* mean, const float* rstd, void* dx, void* dw, void* db,
                                void* workspace, hipStream_t stream);

// ----------------------------------------------------------------------------
// Vocabulary losses: cross entropy (top == 0) and distillation.
// ----------------------------------------------------------------------------
struct LossProblem {
  const void* x;           // [rows, hidden]
  int64_t rows, hidden, vocab;
  bdr_dtype dt;
  const void* w;           // [vocab, hidden]
  const void* w1;          // [vocab, rank]
  const void* w2;
  int rank;
  const int32_t* prev;     // [rows]
  const int32_t* labels;   // cross entropy [rows]
  int top;                 // distillation: teacher entries per row
  const int32_t* ids;      // [rows, top]
  const void* u;           // [rows, top]
  bdr_dtype u_dt;
  float temperature;       // 1 for cross entropy
};
struct LossGrads {         // each may be NULL
  void* hidden;
  void* w;
  void* w1;
  void* w2;
};
size_t loss_workspace(const LossProblem& p, bool backward);
hipError_t launch_loss_forward(const LossProblem& p, void* workspace, float* loss, float* lse,
                               float* picked, hipStream_t stream);
hipError_t launch_loss_backward(const LossProblem& p, const LossGrads& out, void* workspace,
                                const float* lse, const float* picked, const float* loss_grad,
                                hipStream_t stream);
// zero fill of bytes % 16 == 0 with vector stores
hipError_t launch_clear(void* p, int64_t bytes, hipStream_t stream);
// the gradients of a call without rows: zeros
hipError_t launch_loss_clear(const LossProblem& p, const LossGrads& out, hipStream_t stream);

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace bdr
