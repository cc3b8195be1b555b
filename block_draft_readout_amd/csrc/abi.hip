// C ABI of libbdr: argument validation, workspace sizing and dispatch to the
// gfx950 kernel launchers.  Every host-checkable argument is validated before
// anything is enqueued; the device architecture is checked once per device.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "bdr_internal.h"

using namespace bdr;

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

int hip_fail(hipError_t e, const char* what) {
  return fail(BDR_EHIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool valid_dtype(int dt) { return dt == BDR_F32 || dt == BDR_BF16; }
// calls with a GEMM weight also take the packed bf16 layout
bool valid_gemm_dtype(int dt) { return valid_dtype(dt) || dt == BDR_BF16_PACKED; }

constexpr int64_t kMaxVocab = 0x7FFFFFFELL;
constexpr int64_t kMaxElems = int64_t(1) << 40;  // per tensor; keeps index math in range
constexpr int64_t kMaxBytes = 0x7FFFFFFFLL;      // per buffer resource
constexpr int64_t kMaxMarkovVocab = int64_t(1) << 21;

// 0 unknown, 1 gfx950, 2 other; compute units per device
int g_dev_state[256];
int g_dev_cus[256];
std::mutex g_dev_mu;

// Checks that the current device is gfx950; *cus receives its compute-unit count.
int check_device(int* cus = nullptr) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= 256) return fail(BDR_EUNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (g_dev_state[dev] == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDeviceProperties");
    g_dev_state[dev] = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_dev_cus[dev] = prop.multiProcessorCount;
    if (g_dev_state[dev] == 2)
      return fail(BDR_EUNSUPPORTED, "device %d is %s; libbdr is built for gfx950 only", dev,
                  prop.gcnArchName);
  }
  if (g_dev_state[dev] != 1)
    return fail(BDR_EUNSUPPORTED, "device %d is not gfx950; libbdr is built for gfx950 only", dev);
  if (cus) *cus = g_dev_cus[dev];
  return BDR_OK;
}

int need_ptr(const void* p, const char* name, size_t align = 16) {
  if (!p) return fail(BDR_EINVAL, "%s must not be NULL", name);
  if (!aligned(p, align)) return fail(BDR_EINVAL, "%s must be %zu-byte aligned", name, align);
  return BDR_OK;
}

int need_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return BDR_OK;
  if (!ws) return fail(BDR_EWORKSPACE, "workspace of %zu bytes required, got NULL", need);
  if (!aligned(ws, 256)) return fail(BDR_EWORKSPACE, "workspace must be 256-byte aligned");
  if (have < need) return fail(BDR_EWORKSPACE, "workspace of %zu bytes required, got %zu", need, have);
  return BDR_OK;
}

#define BDR_TRY(x)               \
  do {                           \
    const int rc_ = (x);         \
    if (rc_ != BDR_OK) return rc_; \
  } while (0)

int fc_shape(int64_t rows, int64_t hidden, int n_taps, int wdt) {
  if (!valid_gemm_dtype(wdt)) return fail(BDR_EINVAL, "unknown dtype %d", wdt);
  const int dt = act_dtype(static_cast<bdr_dtype>(wdt));
  if (n_taps < 1) return fail(BDR_EINVAL, "n_taps must be >= 1, got %d", n_taps);
  if (n_taps > BDR_MAX_TAPS) return fail(BDR_EUNSUPPORTED, "n_taps %d > %d", n_taps, BDR_MAX_TAPS);
  if (rows < 0) return fail(BDR_EINVAL, "rows must be >= 0");
  if (hidden <= 0) return fail(BDR_EINVAL, "hidden must be > 0");
  const int ks = dt == BDR_BF16 ? 32 : 16;
  if (hidden % ks)
    return fail(BDR_EUNSUPPORTED, "hidden %lld must be a multiple of %d for this dtype",
                static_cast<long long>(hidden), ks);
  // each tap [rows, H] and each 64-row slab of fc_w must stay below 2^31 bytes
  const int64_t es = dt == BDR_BF16 ? 2 : 4;
  if (rows > kMaxBytes / (hidden * es) || hidden * n_taps > kMaxBytes / (64 * es))
    return fail(BDR_EUNSUPPORTED, "fc problem too large (per-operand byte limit 2^31)");
  if (wdt == BDR_BF16_PACKED) {
    if (n_taps > 1 && hidden % 128)
      return fail(BDR_EUNSUPPORTED, "a multi-tap fc with packed weights needs hidden %% 128 == 0");
    if (packed_weight_bytes(hidden, hidden * n_taps) == 0)
      return fail(BDR_EUNSUPPORTED, "packed fc_w would reach 2^31 bytes");
  }
  return BDR_OK;
}

int lm_shape(int64_t rows, int64_t hidden, int64_t vocab, int wdt) {
  if (!valid_gemm_dtype(wdt)) return fail(BDR_EINVAL, "unknown dtype %d", wdt);
  const int dt = act_dtype(static_cast<bdr_dtype>(wdt));
  if (rows < 0) return fail(BDR_EINVAL, "rows must be >= 0");
  if (hidden <= 0) return fail(BDR_EINVAL, "hidden must be > 0");
  if (vocab <= 0) return fail(BDR_EINVAL, "vocab must be > 0");
  if (vocab > kMaxVocab) return fail(BDR_EUNSUPPORTED, "vocab must be < 2^31 - 1");
  const int e = dt == BDR_BF16 ? 8 : 4;
  if (hidden % e)
    return fail(BDR_EUNSUPPORTED, "hidden %lld must be a multiple of %d for this dtype",
                static_cast<long long>(hidden), e);
  const int64_t es = dt == BDR_BF16 ? 2 : 4;
  if (rows > kMaxBytes / (hidden * es) || hidden > kMaxBytes / (64 * es) ||
      vocab > kMaxElems / hidden || rows > kMaxElems / vocab)
    return fail(BDR_EUNSUPPORTED, "LM-head problem too large (per-operand byte limit 2^31)");
  if (wdt == BDR_BF16_PACKED) {
    if (packed_weight_bytes(vocab, hidden) == 0)
      return fail(BDR_EUNSUPPORTED, "packed lm_head_w would reach 2^31 bytes");
    // a slab's logits are addressed with 32-bit offsets
    if (std::min<int64_t>(rows, kPackedSlabRows) * vocab * 4 >= (int64_t(1) << 32))
      return fail(BDR_EUNSUPPORTED, "LM head with packed weights: vocab too large");
  }
  return BDR_OK;
}

int block_shape(int64_t batch, int k, int64_t vocab) {
  if (batch < 0) return fail(BDR_EINVAL, "batch must be >= 0");
  if (k < 1) return fail(BDR_EINVAL, "k must be >= 1, got %d", k);
  if (k > BDR_MAX_K) return fail(BDR_EUNSUPPORTED, "k %d > %d", k, BDR_MAX_K);
  if (vocab <= 0) return fail(BDR_EINVAL, "vocab must be > 0");
  if (vocab > kMaxVocab) return fail(BDR_EUNSUPPORTED, "vocab must be < 2^31 - 1");
  if (batch > 0x7FFFFFFFLL / (k + 1)) return fail(BDR_EUNSUPPORTED, "batch too large");
  if (batch * (k + 1) > kMaxElems / vocab) return fail(BDR_EUNSUPPORTED, "block too large");
  return BDR_OK;
}

int markov_shape(int dt, const void* w1, const void* w2, int rank, int64_t vocab, int k) {
  if (!valid_dtype(dt)) return fail(BDR_EINVAL, "unknown dtype %d", dt);
  // logits of 16 rows of one position, and each Markov matrix, under 2^31 bytes
  if (vocab > kMaxMarkovVocab) return fail(BDR_EUNSUPPORTED, "vocab must be <= 2^21 here");
  if (rank < 0) return fail(BDR_EINVAL, "rank must be >= 0");
  if (rank > BDR_MAX_RANK) return fail(BDR_EUNSUPPORTED, "rank %d > %d", rank, BDR_MAX_RANK);
  if ((w1 == nullptr) != (w2 == nullptr))
    return fail(BDR_EINVAL, "markov_w1 and markov_w2 must both be given or both be NULL");
  if (w1 && rank > 0) {
    const int e = dt == BDR_BF16 ? 8 : 4;
    if (rank % e) return fail(BDR_EUNSUPPORTED, "rank %d must be a multiple of %d for this dtype", rank, e);
    BDR_TRY(need_ptr(w1, "markov_w1"));
    BDR_TRY(need_ptr(w2, "markov_w2"));
  }
  return BDR_OK;
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// ---------------------------------------------------------------------------- no-allocation scratch
// The Markov hand-off workspace of dspark_draft_block_noalloc.  Each device the
// library runs on holds its own copy of this array until the process ends (zero
// when the code object is loaded).  In host code `scratch` names a host-side
// stand-in, not device memory: its device address is taken once per device with
// hipGetSymbolAddress (that device current) and only that address is passed on.
static __device__ __align__(256) unsigned char scratch[BDR_NOALLOC_SCRATCH_BYTES];
void* g_scratch_ptr[256];
std::mutex g_scratch_mu;

int scratch_address(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= 256) return fail(BDR_EUNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return hip_fail(e, "hipGetSymbolAddress(scratch)");
    if (!p) return fail(BDR_EHIP, "hipGetSymbolAddress(scratch) returned NULL");
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return BDR_OK;
}

// zero-fills n bytes (n % 16 == 0) with vector stores: the hand-off slots and
// counters must start at zero, whatever an earlier call on this device left
__global__ __launch_bounds__(256) void zero_fill_kernel(uint4* p, size_t n16) {
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n16;
       i += static_cast<size_t>(gridDim.x) * 256)
    p[i] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace

extern "C" {

int bdr_abi_version(void) { return 11; }

void bdr_set_markov_poll_timeout_us(double us) { bdr::set_poll_timeout_us(us); }

void bdr_set_markov_forced_time_out(int on) { bdr::set_forced_time_out(on != 0); }

int bdr_set_row_split_override(int ring, int64_t workgroups, int ksplit) {
  if (ring < 0 || workgroups < 0 || ksplit < 0 || workgroups > (int64_t(1) << 20) || ksplit > 256)
    return fail(BDR_EINVAL, "row-split override: ring %d, workgroups %lld, ksplit %d out of range",
                ring, static_cast<long long>(workgroups), ksplit);
  bdr::set_row_split_override(ring, workgroups, ksplit);
  return BDR_OK;
}

const char* bdr_last_error(void) { return g_err; }

// ---------------------------------------------------------------------------- packed weights
size_t bdr_packed_weight_bytes(int64_t rows, int64_t cols) {
  return packed_weight_bytes(rows, cols);
}

int bdr_pack_weight(const void* w, int64_t rows, int64_t cols, void* packed, void* stream) {
  const size_t bytes = packed_weight_bytes(rows, cols);
  if (bytes == 0)
    return fail(BDR_EUNSUPPORTED, "weight [%lld, %lld] cannot be packed (cols %% 8 == 0 and a "
                "packed copy under 2^31 bytes are required)", static_cast<long long>(rows),
                static_cast<long long>(cols));
  BDR_TRY(need_ptr(w, "w"));
  BDR_TRY(need_ptr(packed, "packed"));
  const uintptr_t w0 = reinterpret_cast<uintptr_t>(w), p0 = reinterpret_cast<uintptr_t>(packed);
  const uintptr_t wbytes = static_cast<uintptr_t>(rows) * static_cast<uintptr_t>(cols) * 2;
  if (w0 < p0 + bytes && p0 < w0 + wbytes) return fail(BDR_EINVAL, "packed overlaps w");
  BDR_TRY(check_device());
  const hipError_t e = launch_pack_weight(w, rows, cols, packed, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "bdr_pack_weight launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S1
size_t dflash_fuse_fc_workspace_bytes(int64_t rows, int64_t hidden, int n_taps, bdr_dtype dt) {
  if (fc_shape(rows, hidden, n_taps, dt) != BDR_OK || rows == 0) return 0;
  return plan_gemm(rows, hidden, hidden * n_taps, dt, true, n_taps).workspace;
}

int dflash_fuse_fc(const void* const* taps, int n_taps, int64_t rows, int64_t hidden,
                   bdr_dtype dt, const void* fc_w, void* out, void* workspace,
                   size_t workspace_bytes, void* stream) {
  BDR_TRY(fc_shape(rows, hidden, n_taps, dt));
  if (rows == 0) return BDR_OK;
  if (!taps) return fail(BDR_EINVAL, "taps must not be NULL");
  for (int t = 0; t < n_taps; ++t) {
    if (!taps[t]) return fail(BDR_EINVAL, "taps[%d] must not be NULL", t);
    if (!aligned(taps[t], 16)) return fail(BDR_EINVAL, "taps[%d] must be 16-byte aligned", t);
  }
  BDR_TRY(need_ptr(fc_w, "fc_w"));
  BDR_TRY(need_ptr(out, "out"));
  const GemmPlan p = plan_gemm(rows, hidden, hidden * n_taps, dt, true, n_taps);
  BDR_TRY(need_ws(workspace, workspace_bytes, p.workspace));
  BDR_TRY(check_device());
  hipError_t e = launch_gemm(p, dt, taps, n_taps, hidden, rows, hidden, fc_w, out,
                             act_dtype(dt) == BDR_BF16 ? OUT_BF16 : OUT_F32, workspace,
                             as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dflash_fuse_fc launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S1 + S2 in one launch
namespace {
// the pair plan when both GEMMs take it (bf16, row-split shapes), else !ok
PairPlan fc_lm_pair(int64_t rows, int64_t hidden, int n_taps, int64_t lm_rows, int64_t vocab,
                    bdr_dtype dt) {
  if (act_dtype(dt) != BDR_BF16 || rows == 0 || lm_rows == 0) return PairPlan{};
  return plan_gemm_pair(lm_rows, vocab, hidden, rows, hidden, hidden * n_taps, n_taps,
                        dt == BDR_BF16_PACKED);
}
}  // namespace

size_t dflash_fuse_fc_lm_head_workspace_bytes(int64_t rows, int64_t hidden, int n_taps,
                                              int64_t lm_rows, int64_t vocab, bdr_dtype dt) {
  if (fc_shape(rows, hidden, n_taps, dt) != BDR_OK ||
      lm_shape(lm_rows, hidden, vocab, dt) != BDR_OK)
    return 0;
  const PairPlan pp = fc_lm_pair(rows, hidden, n_taps, lm_rows, vocab, dt);
  if (pp.ok) return pp.workspace;
  return rows == 0 ? 0 : plan_gemm(rows, hidden, hidden * n_taps, dt, true, n_taps).workspace;
}

int dflash_fuse_fc_lm_head(const void* const* taps, int n_taps, int64_t rows, int64_t hidden,
                           bdr_dtype dt, const void* fc_w, void* fc_out, const void* lm_hidden,
                           int64_t lm_rows, int64_t vocab, const void* lm_head_w, float* logits,
                           void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(fc_shape(rows, hidden, n_taps, dt));
  BDR_TRY(lm_shape(lm_rows, hidden, vocab, dt));
  if (rows > 0) {
    if (!taps) return fail(BDR_EINVAL, "taps must not be NULL");
    for (int t = 0; t < n_taps; ++t) {
      if (!taps[t]) return fail(BDR_EINVAL, "taps[%d] must not be NULL", t);
      if (!aligned(taps[t], 16)) return fail(BDR_EINVAL, "taps[%d] must be 16-byte aligned", t);
    }
    BDR_TRY(need_ptr(fc_w, "fc_w"));
    BDR_TRY(need_ptr(fc_out, "fc_out"));
  }
  if (lm_rows > 0) {
    BDR_TRY(need_ptr(lm_hidden, "lm_hidden"));
    BDR_TRY(need_ptr(lm_head_w, "lm_head_w"));
    BDR_TRY(need_ptr(logits, "logits"));
  }
  if (rows == 0 && lm_rows == 0) return BDR_OK;
  const PairPlan pp = fc_lm_pair(rows, hidden, n_taps, lm_rows, vocab, dt);
  const GemmPlan pf = rows > 0 && !pp.ok ? plan_gemm(rows, hidden, hidden * n_taps, dt, true, n_taps)
                                         : GemmPlan{};
  BDR_TRY(need_ws(workspace, workspace_bytes, pp.ok ? pp.workspace : pf.workspace));
  BDR_TRY(check_device());
  const hipStream_t st = as_stream(stream);
  hipError_t e;
  if (pp.ok) {
    e = launch_gemm_pair(pp, lm_hidden, lm_head_w, logits, taps, n_taps, hidden, fc_w, fc_out,
                         workspace, dt == BDR_BF16_PACKED, st);
    if (e != hipSuccess) return hip_fail(e, "dflash_fuse_fc_lm_head launch");
    return BDR_OK;
  }
  if (rows > 0) {
    e = launch_gemm(pf, dt, taps, n_taps, hidden, rows, hidden, fc_w, fc_out,
                    act_dtype(dt) == BDR_BF16 ? OUT_BF16 : OUT_F32, workspace, st);
    if (e != hipSuccess) return hip_fail(e, "dflash_fuse_fc_lm_head fc launch");
  }
  if (lm_rows > 0) {
    const GemmPlan pl = plan_gemm(lm_rows, vocab, hidden, dt, false);
    const void* a[1] = {lm_hidden};
    e = launch_gemm(pl, dt, a, 1, hidden, lm_rows, vocab, lm_head_w, logits, OUT_F32, nullptr, st);
    if (e != hipSuccess) return hip_fail(e, "dflash_fuse_fc_lm_head LM-head launch");
  }
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S2
int dspark_lm_head(const void* hidden, int64_t rows, int64_t hidden_size, int64_t vocab,
                   bdr_dtype dt, const void* lm_head_w, float* logits, void* stream) {
  BDR_TRY(lm_shape(rows, hidden_size, vocab, dt));
  if (rows == 0) return BDR_OK;
  BDR_TRY(need_ptr(hidden, "hidden"));
  BDR_TRY(need_ptr(lm_head_w, "lm_head_w"));
  BDR_TRY(need_ptr(logits, "logits"));
  BDR_TRY(check_device());
  const GemmPlan p = plan_gemm(rows, vocab, hidden_size, dt, false);
  const void* a[1] = {hidden};
  hipError_t e = launch_gemm(p, dt, a, 1, hidden_size, rows, vocab, lm_head_w, logits, OUT_F32,
                             nullptr, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_lm_head launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S1 taps: hc average
int dflash_hc_average(const void* const* captured, int n_taps, int hc, int64_t rows,
                      int64_t hidden, int64_t stream_stride, int64_t row_stride, bdr_dtype dt,
                      void* const* taps_out, void* stream) {
  if (!valid_dtype(dt)) return fail(BDR_EINVAL, "unknown dtype %d", dt);
  if (n_taps < 1) return fail(BDR_EINVAL, "n_taps must be >= 1, got %d", n_taps);
  if (n_taps > BDR_MAX_TAPS) return fail(BDR_EUNSUPPORTED, "n_taps %d > %d", n_taps, BDR_MAX_TAPS);
  if (hc < 1) return fail(BDR_EINVAL, "hc must be >= 1, got %d", hc);
  if (hc > BDR_MAX_HC) return fail(BDR_EUNSUPPORTED, "hc %d > %d", hc, BDR_MAX_HC);
  if (rows < 0) return fail(BDR_EINVAL, "rows must be >= 0");
  if (hidden <= 0) return fail(BDR_EINVAL, "hidden must be > 0");
  if (hidden % 8) return fail(BDR_EUNSUPPORTED, "hidden must be a multiple of 8");
  if (stream_stride < 0 || row_stride < hidden || stream_stride % 8 || row_stride % 8)
    return fail(BDR_EINVAL, "strides must be multiples of 8 elements, row_stride >= hidden, "
                "stream_stride >= 0");
  if (rows > kMaxElems / hidden || rows > kMaxElems / row_stride || hc > kMaxElems / (stream_stride + 1))
    return fail(BDR_EUNSUPPORTED, "problem too large");
  if (rows == 0) return BDR_OK;
  if (!captured || !taps_out) return fail(BDR_EINVAL, "captured and taps_out must not be NULL");
  for (int t = 0; t < n_taps; ++t) {
    if (!captured[t] || !taps_out[t]) return fail(BDR_EINVAL, "tap %d pointer is NULL", t);
    if (!aligned(captured[t], 16) || !aligned(taps_out[t], 16))
      return fail(BDR_EINVAL, "tap %d pointers must be 16-byte aligned", t);
  }
  BDR_TRY(check_device());
  hipError_t e = launch_hc_average(captured, taps_out, n_taps, hc, rows, hidden, stream_stride,
                                   row_stride, dt, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dflash_hc_average launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S1/S2, fp8 weights
namespace {

// bf16 activations [rows, H] read against E4M3 weights [N, K] with K = n_seg * H
int fp8_shape(int64_t rows, int64_t hidden, int n_seg, int64_t n_out) {
  if (n_seg < 1) return fail(BDR_EINVAL, "n_taps must be >= 1, got %d", n_seg);
  if (n_seg > BDR_MAX_TAPS) return fail(BDR_EUNSUPPORTED, "n_taps %d > %d", n_seg, BDR_MAX_TAPS);
  if (rows < 0) return fail(BDR_EINVAL, "rows must be >= 0");
  if (hidden <= 0) return fail(BDR_EINVAL, "hidden must be > 0");
  if (n_out <= 0) return fail(BDR_EINVAL, "output width must be > 0");
  if (n_out > kMaxVocab) return fail(BDR_EUNSUPPORTED, "output width must be < 2^31 - 1");
  if (hidden % 64)
    return fail(BDR_EUNSUPPORTED, "hidden %lld must be a multiple of 64 for fp8 weights",
                static_cast<long long>(hidden));
  // each activation tensor, and the W rows one workgroup streams (<= 192 rows), under 2^31 bytes
  if (rows > kMaxBytes / (hidden * 2) || hidden * n_seg > kMaxBytes / 192 ||
      n_out > kMaxElems / (hidden * n_seg) || rows > kMaxElems / n_out)
    return fail(BDR_EUNSUPPORTED, "problem too large (per-operand byte limit 2^31)");
  return BDR_OK;
}

}  // namespace

size_t dflash_fuse_fc_fp8_workspace_bytes(int64_t rows, int64_t hidden, int n_taps) {
  if (fp8_shape(rows, hidden, n_taps, hidden) != BDR_OK || rows == 0) return 0;
  return plan_gemm_fp8(rows, hidden, hidden * n_taps, true, n_taps).workspace;
}

int dflash_fuse_fc_fp8(const void* const* taps, int n_taps, int64_t rows, int64_t hidden,
                       const uint8_t* fc_q, const float* fc_scale, void* out, void* workspace,
                       size_t workspace_bytes, void* stream) {
  BDR_TRY(fp8_shape(rows, hidden, n_taps, hidden));
  if (rows == 0) return BDR_OK;
  if (!taps) return fail(BDR_EINVAL, "taps must not be NULL");
  for (int t = 0; t < n_taps; ++t) {
    if (!taps[t]) return fail(BDR_EINVAL, "taps[%d] must not be NULL", t);
    if (!aligned(taps[t], 16)) return fail(BDR_EINVAL, "taps[%d] must be 16-byte aligned", t);
  }
  BDR_TRY(need_ptr(fc_q, "fc_q"));
  BDR_TRY(need_ptr(fc_scale, "fc_scale", 4));
  BDR_TRY(need_ptr(out, "out"));
  const GemmPlan p = plan_gemm_fp8(rows, hidden, hidden * n_taps, true, n_taps);
  if (!p.stream) return fail(BDR_EUNSUPPORTED, "fc shape not supported with fp8 weights");
  BDR_TRY(need_ws(workspace, workspace_bytes, p.workspace));
  BDR_TRY(check_device());
  hipError_t e = launch_gemm_fp8(p, taps, n_taps, hidden, rows, hidden, fc_q, fc_scale, out,
                                 OUT_BF16, workspace, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dflash_fuse_fc_fp8 launch");
  return BDR_OK;
}

int dspark_lm_head_fp8(const void* hidden, int64_t rows, int64_t hidden_size, int64_t vocab,
                       const uint8_t* lm_head_q, const float* lm_head_scale, float* logits,
                       void* stream) {
  BDR_TRY(fp8_shape(rows, hidden_size, 1, vocab));
  if (rows == 0) return BDR_OK;
  BDR_TRY(need_ptr(hidden, "hidden"));
  BDR_TRY(need_ptr(lm_head_q, "lm_head_q"));
  BDR_TRY(need_ptr(lm_head_scale, "lm_head_scale", 4));
  BDR_TRY(need_ptr(logits, "logits"));
  const GemmPlan p = plan_gemm_fp8(rows, vocab, hidden_size, false);
  if (!p.stream) return fail(BDR_EUNSUPPORTED, "LM-head shape not supported with fp8 weights");
  BDR_TRY(check_device());
  const void* a[1] = {hidden};
  hipError_t e = launch_gemm_fp8(p, a, 1, hidden_size, rows, vocab, lm_head_q, lm_head_scale,
                                 logits, OUT_F32, nullptr, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_lm_head_fp8 launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S3
size_t dspark_markov_workspace_bytes(int64_t batch, int k) {
  if (batch < 0 || k < 1 || k > BDR_MAX_K) return 0;
  return markov_workspace(batch, k);
}

int dspark_markov_argmax(const float* logits, int64_t batch, int k, int64_t vocab,
                         bdr_dtype wdt, const void* markov_w1, const void* markov_w2, int rank,
                         const int32_t* prev_token, int32_t* draft_tokens, int32_t* status,
                         void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(block_shape(batch, k, vocab));
  BDR_TRY(markov_shape(wdt, markov_w1, markov_w2, rank, vocab, k));
  if (batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(logits, "logits"));
  BDR_TRY(need_ptr(prev_token, "prev_token", 4));
  BDR_TRY(need_ptr(draft_tokens, "draft_tokens", 4));
  if (status) BDR_TRY(need_ptr(status, "status", 4));
  BDR_TRY(need_ws(workspace, workspace_bytes, markov_workspace(batch, k)));
  int cus = 0;
  BDR_TRY(check_device(&cus));
  hipError_t e = launch_markov(logits, batch, k, vocab, wdt, markov_w1, markov_w2, rank,
                               prev_token, draft_tokens, status, workspace, cus,
                               as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_markov_argmax launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S2+S3
size_t dspark_draft_workspace_bytes(int64_t batch, int k, int64_t vocab, int logits_in_workspace) {
  if (batch < 0 || k < 1 || k > BDR_MAX_K || vocab <= 0 || vocab > kMaxVocab) return 0;
  size_t n = markov_workspace(batch, k);
  if (logits_in_workspace) n += align256(static_cast<size_t>(batch) * k * vocab * 4);
  return n;
}

int dspark_draft_block(const void* draft_hidden, int64_t batch, int k, int64_t hidden,
                       int64_t vocab, bdr_dtype dt, const void* lm_head_w, const void* markov_w1,
                       const void* markov_w2, int rank, const int32_t* prev_token,
                       int32_t* draft_tokens, float* logits_out, int32_t* status,
                       void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(block_shape(batch, k, vocab));
  BDR_TRY(lm_shape(batch * k, hidden, vocab, dt));
  BDR_TRY(markov_shape(act_dtype(dt), markov_w1, markov_w2, rank, vocab, k));
  if (batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(draft_hidden, "draft_hidden"));
  BDR_TRY(need_ptr(lm_head_w, "lm_head_w"));
  BDR_TRY(need_ptr(prev_token, "prev_token", 4));
  BDR_TRY(need_ptr(draft_tokens, "draft_tokens", 4));
  if (logits_out) BDR_TRY(need_ptr(logits_out, "logits_out"));
  if (status) BDR_TRY(need_ptr(status, "status", 4));
  const size_t need = dspark_draft_workspace_bytes(batch, k, vocab, logits_out == nullptr);
  BDR_TRY(need_ws(workspace, workspace_bytes, need));
  int cus = 0;
  BDR_TRY(check_device(&cus));
  char* ws = static_cast<char*>(workspace);
  float* logits = logits_out;
  if (!logits) {
    logits = reinterpret_cast<float*>(ws);
    ws += align256(static_cast<size_t>(batch) * k * vocab * 4);
  }
  const GemmPlan p = plan_gemm(batch * k, vocab, hidden, dt, false);
  const void* a[1] = {draft_hidden};
  hipError_t e = launch_gemm(p, dt, a, 1, hidden, batch * k, vocab, lm_head_w, logits, OUT_F32,
                             nullptr, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_draft_block LM-head launch");
  e = launch_markov(logits, batch, k, vocab, act_dtype(dt), markov_w1, markov_w2, rank,
                    prev_token, draft_tokens, status, ws, cus, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_draft_block Markov launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S2+S3, no allocation
int dspark_draft_block_noalloc(const void* draft_hidden, int64_t batch, int k, int64_t hidden,
                               int64_t vocab, bdr_dtype dt, const void* lm_head_w,
                               const void* markov_w1, const void* markov_w2, int rank,
                               const int32_t* prev_token, int32_t* draft_tokens,
                               float* logits_out, int32_t* status, void* stream) {
  BDR_TRY(block_shape(batch, k, vocab));
  BDR_TRY(lm_shape(batch * k, hidden, vocab, dt));
  BDR_TRY(markov_shape(act_dtype(dt), markov_w1, markov_w2, rank, vocab, k));
  const size_t need = markov_workspace(batch, k);
  if (need > BDR_NOALLOC_SCRATCH_BYTES)
    return fail(BDR_EUNSUPPORTED,
                "batch %lld x k %d needs %zu bytes of hand-off scratch; the static scratch "
                "holds %d (batch * k <= 256)", static_cast<long long>(batch), k, need,
                BDR_NOALLOC_SCRATCH_BYTES);
  if (batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(draft_hidden, "draft_hidden"));
  BDR_TRY(need_ptr(lm_head_w, "lm_head_w"));
  BDR_TRY(need_ptr(prev_token, "prev_token", 4));
  BDR_TRY(need_ptr(draft_tokens, "draft_tokens", 4));
  BDR_TRY(need_ptr(logits_out, "logits_out"));
  if (status) BDR_TRY(need_ptr(status, "status", 4));
  int cus = 0;
  BDR_TRY(check_device(&cus));
  void* ws = nullptr;
  BDR_TRY(scratch_address(&ws));
  const GemmPlan p = plan_gemm(batch * k, vocab, hidden, dt, false);
  if (p.workspace != 0) return fail(BDR_EUNSUPPORTED, "LM-head plan needs a workspace");
  const hipStream_t st = as_stream(stream);
  const size_t n16 = need / 16;
  hipLaunchKernelGGL(zero_fill_kernel, dim3(static_cast<unsigned>(std::min<size_t>((n16 + 255) / 256, 1024))),
                     dim3(256), 0, st, static_cast<uint4*>(ws), n16);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "dspark_draft_block_noalloc scratch clear");
  const void* a[1] = {draft_hidden};
  e = launch_gemm(p, dt, a, 1, hidden, batch * k, vocab, lm_head_w, logits_out, OUT_F32, nullptr,
                  st);
  if (e != hipSuccess) return hip_fail(e, "dspark_draft_block_noalloc LM-head launch");
  e = launch_markov(logits_out, batch, k, vocab, act_dtype(dt), markov_w1, markov_w2, rank,
                    prev_token, draft_tokens, status, ws, cus, st);
  if (e != hipSuccess) return hip_fail(e, "dspark_draft_block_noalloc Markov launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- S4
size_t spec_verify_workspace_bytes(int64_t batch, int k, int64_t vocab) {
  if (batch < 0 || k < 1 || k > BDR_MAX_K || vocab <= 0 || vocab > kMaxVocab) return 0;
  return verify_workspace(batch, k, vocab);
}

int spec_verify_greedy(const void* target_logits, bdr_dtype dt, int64_t batch, int k,
                       int64_t vocab, const int32_t* draft_tokens, const float* confidence,
                       float threshold, int32_t* block_len, int32_t* accepted, int32_t* bonus,
                       int32_t* target_argmax, int64_t* accept_counts, int64_t* proposed_counts,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dt)) return fail(BDR_EINVAL, "unknown dtype %d", dt);
  BDR_TRY(block_shape(batch, k, vocab));
  if (batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(target_logits, "target_logits"));
  BDR_TRY(need_ptr(draft_tokens, "draft_tokens", 4));
  if (confidence) BDR_TRY(need_ptr(confidence, "confidence", 4));
  BDR_TRY(need_ptr(block_len, "block_len", 4));
  BDR_TRY(need_ptr(accepted, "accepted", 4));
  BDR_TRY(need_ptr(bonus, "bonus", 4));
  if (target_argmax) BDR_TRY(need_ptr(target_argmax, "target_argmax", 4));
  if (accept_counts) BDR_TRY(need_ptr(accept_counts, "accept_counts", 8));
  if (proposed_counts) BDR_TRY(need_ptr(proposed_counts, "proposed_counts", 8));
  BDR_TRY(need_ws(workspace, workspace_bytes, verify_workspace(batch, k, vocab)));
  BDR_TRY(check_device());
  hipError_t e = launch_verify(target_logits, dt, batch, k, vocab, draft_tokens, confidence,
                               threshold, block_len, accepted, bonus, target_argmax,
                               accept_counts, proposed_counts, workspace, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "spec_verify_greedy launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- sampling
int dspark_gumbel_noise(int64_t batch, int k, int64_t vocab, uint64_t seed, int stream_id,
                        float* noise, void* stream) {
  BDR_TRY(block_shape(batch, k, vocab));
  if (vocab > kMaxMarkovVocab) return fail(BDR_EUNSUPPORTED, "vocab must be <= 2^21 here");
  if (stream_id < 0) return fail(BDR_EINVAL, "stream_id must be >= 0");
  if (batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(noise, "noise", 4));
  BDR_TRY(check_device());
  hipError_t e = launch_gumbel_noise(noise, batch, k, vocab, seed,
                                     static_cast<uint32_t>(stream_id), as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_gumbel_noise launch");
  return BDR_OK;
}

static int need_temperature(float t) {
  if (!(t > 0.f) || !std::isfinite(t)) return fail(BDR_EINVAL, "temperature must be finite and > 0");
  if (!std::isfinite(1.0f / t)) return fail(BDR_EUNSUPPORTED, "temperature too small");
  return BDR_OK;
}

size_t dspark_markov_sample_workspace_bytes(int64_t batch, int k, int64_t vocab) {
  if (batch < 0 || k < 1 || k > BDR_MAX_K || vocab <= 0 || vocab > kMaxMarkovVocab) return 0;
  return markov_sample_workspace(batch, k, vocab);
}

int dspark_markov_sample(const float* logits, int64_t batch, int k, int64_t vocab,
                         bdr_dtype wdt, const void* markov_w1, const void* markov_w2, int rank,
                         const int32_t* prev_token, float temperature, uint64_t seed,
                         int32_t* draft_tokens, float* draft_logits, const float* confidence,
                         float threshold, int32_t* status, void* workspace,
                         size_t workspace_bytes, void* stream) {
  BDR_TRY(block_shape(batch, k, vocab));
  BDR_TRY(markov_shape(wdt, markov_w1, markov_w2, rank, vocab, k));
  BDR_TRY(need_temperature(temperature));
  if (batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(logits, "logits"));
  BDR_TRY(need_ptr(prev_token, "prev_token", 4));
  BDR_TRY(need_ptr(draft_tokens, "draft_tokens", 4));
  BDR_TRY(need_ptr(draft_logits, "draft_logits"));
  if (confidence) BDR_TRY(need_ptr(confidence, "confidence", 4));
  if (status) BDR_TRY(need_ptr(status, "status", 4));
  BDR_TRY(need_ws(workspace, workspace_bytes, markov_sample_workspace(batch, k, vocab)));
  int cus = 0;
  BDR_TRY(check_device(&cus));
  hipError_t e = launch_markov_sample(logits, batch, k, vocab, wdt, markov_w1, markov_w2, rank,
                                      prev_token, 1.0f / temperature, seed, draft_tokens,
                                      draft_logits, confidence, threshold, status, workspace, cus,
                                      as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_markov_sample launch");
  return BDR_OK;
}

size_t spec_verify_sample_workspace_bytes(int64_t batch, int k, int64_t vocab) {
  if (batch < 0 || k < 1 || k > BDR_MAX_K || vocab <= 0 || vocab > kMaxVocab) return 0;
  return sample_verify_workspace(batch, k, vocab);
}

int spec_verify_sample(const void* target_logits, bdr_dtype dt, int64_t batch, int k,
                       int64_t vocab, const int32_t* draft_tokens, const float* draft_logits,
                       const float* confidence, float threshold, float temperature, uint64_t seed,
                       int32_t* block_len, int32_t* accepted, int32_t* bonus,
                       int64_t* accept_counts, int64_t* proposed_counts, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dt)) return fail(BDR_EINVAL, "unknown dtype %d", dt);
  BDR_TRY(block_shape(batch, k, vocab));
  BDR_TRY(need_temperature(temperature));
  if (batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(target_logits, "target_logits"));
  BDR_TRY(need_ptr(draft_tokens, "draft_tokens", 4));
  BDR_TRY(need_ptr(draft_logits, "draft_logits"));
  if (confidence) BDR_TRY(need_ptr(confidence, "confidence", 4));
  BDR_TRY(need_ptr(block_len, "block_len", 4));
  BDR_TRY(need_ptr(accepted, "accepted", 4));
  BDR_TRY(need_ptr(bonus, "bonus", 4));
  if (accept_counts) BDR_TRY(need_ptr(accept_counts, "accept_counts", 8));
  if (proposed_counts) BDR_TRY(need_ptr(proposed_counts, "proposed_counts", 8));
  BDR_TRY(need_ws(workspace, workspace_bytes, sample_verify_workspace(batch, k, vocab)));
  BDR_TRY(check_device());
  hipError_t e = launch_verify_sample(target_logits, dt, batch, k, vocab, draft_tokens,
                                      draft_logits, confidence, threshold, 1.0f / temperature,
                                      seed, block_len, accepted, bonus, accept_counts,
                                      proposed_counts, workspace, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "spec_verify_sample launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- loop
int spec_commit(const int32_t* draft_tokens, const int32_t* accepted, const int32_t* bonus,
                const int32_t* block_len, int64_t batch, int k, int32_t* next_prev,
                int32_t* emitted, int32_t* draft_list, int32_t* row_index, int32_t* row_count,
                int32_t* row_offsets, void* stream) {
  if (batch < 0) return fail(BDR_EINVAL, "batch must be >= 0");
  if (k < 1) return fail(BDR_EINVAL, "k must be >= 1, got %d", k);
  if (k > BDR_MAX_K) return fail(BDR_EUNSUPPORTED, "k %d > %d", k, BDR_MAX_K);
  if (batch > 0x7FFFFFFFLL / (k + 1)) return fail(BDR_EUNSUPPORTED, "batch too large");
  if (batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(draft_tokens, "draft_tokens", 4));
  BDR_TRY(need_ptr(accepted, "accepted", 4));
  BDR_TRY(need_ptr(bonus, "bonus", 4));
  if (block_len) BDR_TRY(need_ptr(block_len, "block_len", 4));
  BDR_TRY(need_ptr(next_prev, "next_prev", 4));
  for (const int32_t* p : {static_cast<const int32_t*>(emitted), static_cast<const int32_t*>(draft_list),
                           static_cast<const int32_t*>(row_index), static_cast<const int32_t*>(row_count),
                           static_cast<const int32_t*>(row_offsets)})
    if (p) BDR_TRY(need_ptr(p, "output", 4));
  BDR_TRY(check_device());
  hipError_t e = launch_commit(draft_tokens, accepted, bonus, block_len, batch, k, next_prev,
                               emitted, draft_list, row_index, row_count, row_offsets,
                               as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "spec_commit launch");
  return BDR_OK;
}

size_t dflash_fuse_fc_rows_workspace_bytes(int64_t max_rows, int64_t hidden, int n_taps,
                                           bdr_dtype dt) {
  if (fc_shape(max_rows, hidden, n_taps, dt) != BDR_OK) return 0;
  return fc_rows_workspace(max_rows, hidden, n_taps, dt);
}

int dflash_fuse_fc_rows(const void* const* taps, int n_taps, int64_t rows, int64_t hidden,
                        bdr_dtype dt, const int32_t* row_index, const int32_t* row_count,
                        int64_t max_rows, const void* fc_w, void* out, void* workspace,
                        size_t workspace_bytes, void* stream) {
  BDR_TRY(fc_shape(max_rows, hidden, n_taps, dt));
  BDR_TRY(fc_shape(rows, hidden, n_taps, dt));
  if (max_rows == 0) return BDR_OK;
  if (!taps) return fail(BDR_EINVAL, "taps must not be NULL");
  for (int t = 0; t < n_taps; ++t) {
    if (rows > 0 && !taps[t]) return fail(BDR_EINVAL, "taps[%d] must not be NULL", t);
    if (!aligned(taps[t], 16)) return fail(BDR_EINVAL, "taps[%d] must be 16-byte aligned", t);
  }
  BDR_TRY(need_ptr(row_index, "row_index", 4));
  BDR_TRY(need_ptr(row_count, "row_count", 4));
  BDR_TRY(need_ptr(fc_w, "fc_w"));
  BDR_TRY(need_ptr(out, "out"));
  BDR_TRY(need_ws(workspace, workspace_bytes, fc_rows_workspace(max_rows, hidden, n_taps, dt)));
  BDR_TRY(check_device());
  hipError_t e = launch_fc_rows(taps, n_taps, rows, hidden, dt, row_index, row_count, max_rows,
                                fc_w, out, workspace, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dflash_fuse_fc_rows launch");
  return BDR_OK;
}

size_t dflash_fuse_fc_rows_fp8_workspace_bytes(int64_t max_rows, int64_t hidden, int n_taps) {
  if (fp8_shape(max_rows, hidden, n_taps, hidden) != BDR_OK) return 0;
  return fc_rows_fp8_workspace(max_rows, hidden, n_taps);
}

int dflash_fuse_fc_rows_fp8(const void* const* taps, int n_taps, int64_t rows, int64_t hidden,
                            const int32_t* row_index, const int32_t* row_count, int64_t max_rows,
                            const uint8_t* fc_q, const float* fc_scale, void* out,
                            void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(fp8_shape(max_rows, hidden, n_taps, hidden));
  BDR_TRY(fp8_shape(rows, hidden, n_taps, hidden));
  if (max_rows == 0) return BDR_OK;
  if (!taps) return fail(BDR_EINVAL, "taps must not be NULL");
  for (int t = 0; t < n_taps; ++t) {
    if (rows > 0 && !taps[t]) return fail(BDR_EINVAL, "taps[%d] must not be NULL", t);
    if (!aligned(taps[t], 16)) return fail(BDR_EINVAL, "taps[%d] must be 16-byte aligned", t);
  }
  BDR_TRY(need_ptr(row_index, "row_index", 4));
  BDR_TRY(need_ptr(row_count, "row_count", 4));
  BDR_TRY(need_ptr(fc_q, "fc_q"));
  BDR_TRY(need_ptr(fc_scale, "fc_scale", 4));
  BDR_TRY(need_ptr(out, "out"));
  if (!plan_gemm_fp8(max_rows, hidden, hidden * n_taps, true, n_taps).stream)
    return fail(BDR_EUNSUPPORTED, "fc shape not supported with fp8 weights");
  BDR_TRY(need_ws(workspace, workspace_bytes, fc_rows_fp8_workspace(max_rows, hidden, n_taps)));
  BDR_TRY(check_device());
  hipError_t e = launch_fc_rows_fp8(taps, n_taps, rows, hidden, row_index, row_count, max_rows,
                                    fc_q, fc_scale, out, workspace, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dflash_fuse_fc_rows_fp8 launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- training: row norm
namespace {

constexpr int64_t kMaxNormRows = int64_t(1) << 24;   // 256 work-items each in a 32-bit grid

int norm_shape(int64_t rows, int64_t hidden, int dt) {
  if (!valid_dtype(dt)) return fail(BDR_EINVAL, "unknown dtype %d", dt);
  if (rows < 0) return fail(BDR_EINVAL, "rows must be >= 0");
  if (hidden <= 0) return fail(BDR_EINVAL, "hidden must be > 0");
  if (hidden > BDR_MAX_NORM_HIDDEN)
    return fail(BDR_EUNSUPPORTED, "hidden %lld > %d", static_cast<long long>(hidden),
                BDR_MAX_NORM_HIDDEN);
  const int e = dt == BDR_BF16 ? 8 : 4;
  if (hidden % e)
    return fail(BDR_EUNSUPPORTED, "hidden %lld must be a multiple of %d for this dtype",
                static_cast<long long>(hidden), e);
  if (rows >= kMaxNormRows) return fail(BDR_EUNSUPPORTED, "rows must be < 2^24");
  return BDR_OK;
}

int norm_stride(int64_t rows, int64_t hidden, int64_t stride, int dt, const char* name) {
  const int e = dt == BDR_BF16 ? 8 : 4;
  if (stride < hidden || stride % e)
    return fail(BDR_EINVAL, "%s must be a multiple of %d and at least hidden", name, e);
  if (rows > 0 && stride > kMaxElems / rows) return fail(BDR_EUNSUPPORTED, "%s too large", name);
  return BDR_OK;
}

// [p, p + bytes) and [q, q + qbytes) share an address
bool overlap(const void* p, int64_t bytes, const void* q, int64_t qbytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + static_cast<uintptr_t>(qbytes) && b < a + static_cast<uintptr_t>(bytes);
}

// An argument's memory; p NULL: not given.
struct Span {
  const void* p;
  int64_t bytes;
  const char* name;
};

// No output (the workspace is one) shares memory with an input or another output.
int no_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  auto meet = [](const Span& a, const Span& b) {
    return a.p && b.p && overlap(a.p, a.bytes, b.p, b.bytes);
  };
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return fail(BDR_EINVAL, "%s overlaps %s", o->name, i.name);
    for (auto q = o + 1; q != outs.end(); ++q)
      if (meet(*o, *q)) return fail(BDR_EINVAL, "%s overlaps %s", o->name, q->name);
  }
  return BDR_OK;
}

}  // namespace

int dspark_norm(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, bdr_dtype dt,
                const void* weight, const void* bias, float eps, void* y, float* mean,
                float* rstd, void* stream) {
  BDR_TRY(norm_shape(rows, hidden, dt));
  BDR_TRY(norm_stride(rows, hidden, x_stride, dt, "x_stride"));
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(BDR_EINVAL, "eps must be finite and >= 0");
  if (rows == 0) return BDR_OK;
  BDR_TRY(need_ptr(x, "x"));
  BDR_TRY(need_ptr(weight, "weight"));
  if (bias) BDR_TRY(need_ptr(bias, "bias"));
  BDR_TRY(need_ptr(y, "y"));
  if (mean) BDR_TRY(need_ptr(mean, "mean", 4));
  BDR_TRY(need_ptr(rstd, "rstd", 4));
  const int64_t es = dt == BDR_BF16 ? 2 : 4;
  const Span sx{x, ((rows - 1) * x_stride + hidden) * es, "x"};
  const Span sy{y, rows * hidden * es, "y"};
  const Span sm{mean, rows * 4, "mean"}, sr{rstd, rows * 4, "rstd"};
  if (!(x == y && x_stride == hidden) && overlap(x, sx.bytes, y, sy.bytes))
    return fail(BDR_EINVAL, "y overlaps x (only y == x with x_stride == hidden may)");
  BDR_TRY(no_overlap({sy, sm, sr}, {{weight, hidden * es, "weight"}, {bias, hidden * es, "bias"}}));
  BDR_TRY(no_overlap({sm, sr}, {sx}));
  BDR_TRY(check_device());
  const hipError_t e = launch_norm(x, rows, hidden, x_stride, dt, weight, bias, eps, y, mean, rstd,
                                   as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_norm launch");
  return BDR_OK;
}

size_t dspark_norm_backward_workspace_bytes(int64_t rows, int64_t hidden) {
  if (norm_shape(rows, hidden, BDR_F32) != BDR_OK || rows == 0) return 0;
  return norm_workspace(rows, hidden);
}

int dspark_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                         int64_t rows, int64_t hidden, bdr_dtype dt, const void* weight,
                         const float* mean, const float* rstd, void* dx, void* dweight,
                         void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(norm_shape(rows, hidden, dt));
  BDR_TRY(norm_stride(rows, hidden, x_stride, dt, "x_stride"));
  BDR_TRY(norm_stride(rows, hidden, dy_stride, dt, "dy_stride"));
  if (dweight) BDR_TRY(need_ptr(dweight, "dweight"));
  if (dbias) BDR_TRY(need_ptr(dbias, "dbias"));
  const int64_t es = dt == BDR_BF16 ? 2 : 4;
  if (rows == 0) {
    if (!dweight && !dbias) return BDR_OK;
    BDR_TRY(check_device());
    for (void* p : {dweight, dbias})
      if (p) {
        const hipError_t e = launch_clear(p, hidden * es, as_stream(stream));
        if (e != hipSuccess) return hip_fail(e, "dspark_norm_backward clear");
      }
    return BDR_OK;
  }
  if (!dx && !dweight && !dbias) return fail(BDR_EINVAL, "no gradient is wanted");
  BDR_TRY(need_ptr(dy, "dy"));
  BDR_TRY(need_ptr(x, "x"));
  BDR_TRY(need_ptr(weight, "weight"));
  if (mean) BDR_TRY(need_ptr(mean, "mean", 4));
  BDR_TRY(need_ptr(rstd, "rstd", 4));
  if (dx) BDR_TRY(need_ptr(dx, "dx"));
  const size_t need = dweight || dbias ? norm_workspace(rows, hidden) : 0;
  BDR_TRY(need_ws(workspace, workspace_bytes, need));
  const Span sdy{dy, ((rows - 1) * dy_stride + hidden) * es, "dy"};
  const Span sdx{dx, rows * hidden * es, "dx"};
  const Span sdw{dweight, hidden * es, "dweight"}, sdb{dbias, hidden * es, "dbias"};
  const Span sws{need ? workspace : nullptr, static_cast<int64_t>(need), "workspace"};
  if (dx && !(dx == dy && dy_stride == hidden) && overlap(dy, sdy.bytes, dx, sdx.bytes))
    return fail(BDR_EINVAL, "dx overlaps dy (only dx == dy with dy_stride == hidden may)");
  BDR_TRY(no_overlap({sdx, sdw, sdb, sws}, {{x, ((rows - 1) * x_stride + hidden) * es, "x"},
                                            {weight, hidden * es, "weight"},
                                            {mean, rows * 4, "mean"},
                                            {rstd, rows * 4, "rstd"}}));
  BDR_TRY(no_overlap({sdw, sdb, sws}, {sdy}));
  BDR_TRY(check_device());
  const hipError_t e = launch_norm_backward(dy, dy_stride, x, x_stride, rows, hidden, dt, weight,
                                            mean, rstd, dx, dweight, dbias, workspace,
                                            as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_norm_backward launch");
  return BDR_OK;
}

// ---------------------------------------------------------------------------- training: losses
namespace {

constexpr int64_t kMaxLossRows = int64_t(1) << 20;
constexpr int64_t kMaxLossHidden = int64_t(1) << 20;
constexpr int64_t kMaxLossElems = int64_t(1) << 35;   // of each product: grids stay in 32 bits
constexpr float kMinLossTemperature = 1e-4f, kMaxLossTemperature = 1e4f;

// the sizes of a loss call (top == 0: cross entropy)
int loss_shape(int64_t rows, int64_t hidden, int64_t vocab, int rank, int dt, int top, bool distill) {
  if (!valid_dtype(dt)) return fail(BDR_EINVAL, "unknown dtype %d", dt);
  if (rows < 0) return fail(BDR_EINVAL, "rows must be >= 0");
  if (hidden <= 0) return fail(BDR_EINVAL, "hidden must be > 0");
  if (vocab <= 0) return fail(BDR_EINVAL, "vocab must be > 0");
  if (rank < 0) return fail(BDR_EINVAL, "rank must be >= 0");
  if (rows > kMaxLossRows || hidden > kMaxLossHidden || vocab > kMaxMarkovVocab)
    return fail(BDR_EUNSUPPORTED, "rows and hidden must be <= 2^20 and vocab <= 2^21 here");
  if (rows > kMaxLossElems / vocab || hidden > kMaxLossElems / vocab ||
      (rows > 0 && hidden > kMaxLossElems / rows))
    return fail(BDR_EUNSUPPORTED, "rows * vocab, vocab * hidden and rows * hidden must be <= 2^35");
  if (rank > BDR_MAX_RANK) return fail(BDR_EUNSUPPORTED, "rank %d > %d", rank, BDR_MAX_RANK);
  const int e = dt == BDR_BF16 ? 8 : 4;
  if (hidden % e || rank % e)
    return fail(BDR_EUNSUPPORTED, "hidden %lld and rank %d must be multiples of %d for this dtype",
                static_cast<long long>(hidden), rank, e);
  if (distill && top < 1) return fail(BDR_EINVAL, "top must be >= 1, got %d", top);
  if (distill && top > BDR_MAX_TEACHER)
    return fail(BDR_EUNSUPPORTED, "top %d > %d", top, BDR_MAX_TEACHER);
  return BDR_OK;
}

LossProblem loss_sizes(int64_t rows, int64_t hidden, int64_t vocab, int rank, bdr_dtype dt, int top) {
  LossProblem p{};
  p.rows = rows;
  p.hidden = hidden;
  p.vocab = vocab;
  p.rank = rank;
  p.dt = dt;
  p.top = top;
  p.temperature = 1.0f;
  return p;
}

// the tensors every loss call reads
int loss_inputs(const LossProblem& p) {
  BDR_TRY(need_ptr(p.x, "hidden"));
  BDR_TRY(need_ptr(p.w, "lm_head_w"));
  if (p.rank) {
    BDR_TRY(need_ptr(p.w1, "markov_w1"));
    BDR_TRY(need_ptr(p.w2, "markov_w2"));
    BDR_TRY(need_ptr(p.prev, "prev_token", 4));
  }
  if (p.top) {
    BDR_TRY(need_ptr(p.ids, "teacher_ids", 4));
    BDR_TRY(need_ptr(p.u, "teacher_logits", p.u_dt == BDR_BF16 ? 2 : 4));
  } else {
    BDR_TRY(need_ptr(p.labels, "labels", 4));
  }
  return BDR_OK;
}

// No output of a loss call shares memory with what it reads, or with another output.  lse,
// picked and loss_grad are inputs of the backward call (NULL: outputs, or not given).
int loss_overlaps(const LossProblem& p, std::initializer_list<Span> outs, const float* lse,
                  const float* picked, const float* loss_grad) {
  const int64_t es = p.dt == BDR_BF16 ? 2 : 4, us = p.u_dt == BDR_BF16 ? 2 : 4;
  const int64_t head = p.vocab * p.rank * es, list = p.rows * p.top;
  return no_overlap(outs, {{p.x, p.rows * p.hidden * es, "hidden"},
                           {p.w, p.vocab * p.hidden * es, "lm_head_w"},
                           {p.rank ? p.w1 : nullptr, head, "markov_w1"},
                           {p.rank ? p.w2 : nullptr, head, "markov_w2"},
                           {p.rank ? p.prev : nullptr, p.rows * 4, "prev_token"},
                           {p.top ? nullptr : p.labels, p.rows * 4, "labels"},
                           {p.top ? p.ids : nullptr, list * 4, "teacher_ids"},
                           {p.top ? p.u : nullptr, list * us, "teacher_logits"},
                           {lse, p.rows * 4, "lse"},
                           {picked, list * 4, "picked"},
                           {loss_grad, p.rows * 4, "loss_grad"}});
}

int loss_run_forward(const LossProblem& p, float* loss, float* lse, float* picked, void* workspace,
                     size_t workspace_bytes, void* stream, const char* name) {
  if (p.rows == 0) return BDR_OK;
  BDR_TRY(loss_inputs(p));
  BDR_TRY(need_ptr(loss, "loss", 4));
  BDR_TRY(need_ptr(lse, "lse", 4));
  if (p.top) BDR_TRY(need_ptr(picked, "picked", 4));
  const size_t need = loss_workspace(p, false);
  BDR_TRY(need_ws(workspace, workspace_bytes, need));
  BDR_TRY(loss_overlaps(p, {{loss, p.rows * 4, "loss"},
                            {lse, p.rows * 4, "lse"},
                            {p.top ? picked : nullptr, p.rows * p.top * 4, "picked"},
                            {workspace, static_cast<int64_t>(need), "workspace"}},
                        nullptr, nullptr, nullptr));
  BDR_TRY(check_device());
  const hipError_t e = launch_loss_forward(p, workspace, loss, lse, picked, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, name);
  return BDR_OK;
}

int loss_run_backward(const LossProblem& p, const LossGrads& o, const float* lse,
                      const float* picked, const float* loss_grad, void* workspace,
                      size_t workspace_bytes, void* stream, const char* name) {
  if (!p.rank && (o.w1 || o.w2))
    return fail(BDR_EINVAL, "Markov gradients are wanted without a Markov head");
  if (o.hidden && p.rows) BDR_TRY(need_ptr(o.hidden, "d_hidden"));
  if (o.w) BDR_TRY(need_ptr(o.w, "d_lm_head_w"));
  if (o.w1) BDR_TRY(need_ptr(o.w1, "d_markov_w1"));
  if (o.w2) BDR_TRY(need_ptr(o.w2, "d_markov_w2"));
  if (p.rows == 0) {
    if (!o.w && !o.w1 && !o.w2) return BDR_OK;
    BDR_TRY(check_device());
    const hipError_t e = launch_loss_clear(p, o, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, name);
    return BDR_OK;
  }
  if (!o.hidden && !o.w && !o.w1 && !o.w2) return fail(BDR_EINVAL, "no gradient is wanted");
  BDR_TRY(loss_inputs(p));
  BDR_TRY(need_ptr(lse, "lse", 4));
  if (p.top) BDR_TRY(need_ptr(picked, "picked", 4));
  BDR_TRY(need_ptr(loss_grad, "loss_grad", 4));
  const size_t need = loss_workspace(p, true);
  BDR_TRY(need_ws(workspace, workspace_bytes, need));
  const int64_t es = p.dt == BDR_BF16 ? 2 : 4;
  BDR_TRY(loss_overlaps(p, {{o.hidden, p.rows * p.hidden * es, "d_hidden"},
                            {o.w, p.vocab * p.hidden * es, "d_lm_head_w"},
                            {o.w1, p.vocab * p.rank * es, "d_markov_w1"},
                            {o.w2, p.vocab * p.rank * es, "d_markov_w2"},
                            {workspace, static_cast<int64_t>(need), "workspace"}},
                        lse, p.top ? picked : nullptr, loss_grad));
  BDR_TRY(check_device());
  const hipError_t e = launch_loss_backward(p, o, workspace, lse, picked, loss_grad,
                                            as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, name);
  return BDR_OK;
}

// the Markov head of a loss call: both matrices or neither, neither meaning rank 0
int loss_markov(LossProblem& p, const void* w1, const void* w2, const int32_t* prev) {
  if ((w1 == nullptr) != (w2 == nullptr) && p.rank && p.rows)
    return fail(BDR_EINVAL, "markov_w1 and markov_w2 must both be given or both be NULL");
  if (!w1 && !w2 && p.rows) p.rank = 0;
  p.w1 = w1;
  p.w2 = w2;
  p.prev = prev;
  return BDR_OK;
}

}  // namespace

size_t dspark_ce_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab, int rank,
                                 bdr_dtype dt, int backward) {
  if (loss_shape(rows, hidden, vocab, rank, dt, 0, false) != BDR_OK || rows == 0) return 0;
  return loss_workspace(loss_sizes(rows, hidden, vocab, rank, dt, 0), backward != 0);
}

int dspark_ce_loss(const void* hidden, int64_t rows, int64_t hidden_size, int64_t vocab,
                   bdr_dtype dt, const void* lm_head_w, const void* markov_w1,
                   const void* markov_w2, int rank, const int32_t* prev_token,
                   const int32_t* labels, float* loss, float* lse, void* workspace,
                   size_t workspace_bytes, void* stream) {
  BDR_TRY(loss_shape(rows, hidden_size, vocab, rank, dt, 0, false));
  LossProblem p = loss_sizes(rows, hidden_size, vocab, rank, dt, 0);
  BDR_TRY(loss_markov(p, markov_w1, markov_w2, prev_token));
  p.x = hidden;
  p.w = lm_head_w;
  p.labels = labels;
  return loss_run_forward(p, loss, lse, nullptr, workspace, workspace_bytes, stream,
                          "dspark_ce_loss launch");
}

int dspark_ce_backward(const void* hidden, int64_t rows, int64_t hidden_size, int64_t vocab,
                       bdr_dtype dt, const void* lm_head_w, const void* markov_w1,
                       const void* markov_w2, int rank, const int32_t* prev_token,
                       const int32_t* labels, const float* lse, const float* loss_grad,
                       void* d_hidden, void* d_lm_head_w, void* d_markov_w1, void* d_markov_w2,
                       void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(loss_shape(rows, hidden_size, vocab, rank, dt, 0, false));
  LossProblem p = loss_sizes(rows, hidden_size, vocab, rank, dt, 0);
  BDR_TRY(loss_markov(p, markov_w1, markov_w2, prev_token));
  p.x = hidden;
  p.w = lm_head_w;
  p.labels = labels;
  return loss_run_backward(p, LossGrads{d_hidden, d_lm_head_w, d_markov_w1, d_markov_w2}, lse,
                           nullptr, loss_grad, workspace, workspace_bytes, stream,
                           "dspark_ce_backward launch");
}

size_t dspark_distill_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab, int rank,
                                      int top, bdr_dtype dt, int backward) {
  if (loss_shape(rows, hidden, vocab, rank, dt, top, true) != BDR_OK || rows == 0) return 0;
  return loss_workspace(loss_sizes(rows, hidden, vocab, rank, dt, top), backward != 0);
}

namespace {

int distill_problem(LossProblem& p, const void* hidden, const void* lm_head_w,
                    const int32_t* ids, const void* logits, int teacher_dt, float temperature) {
  if (!valid_dtype(teacher_dt)) return fail(BDR_EINVAL, "unknown teacher dtype %d", teacher_dt);
  if (!(temperature >= kMinLossTemperature && temperature <= kMaxLossTemperature))
    return fail(BDR_EINVAL, "temperature must be in [1e-4, 1e4]");
  p.x = hidden;
  p.w = lm_head_w;
  p.ids = ids;
  p.u = logits;
  p.u_dt = static_cast<bdr_dtype>(teacher_dt);
  p.temperature = temperature;
  return BDR_OK;
}

}  // namespace

int dspark_distill_loss(const void* hidden, int64_t rows, int64_t hidden_size, int64_t vocab,
                        bdr_dtype dt, const void* lm_head_w, const void* markov_w1,
                        const void* markov_w2, int rank, const int32_t* prev_token,
                        const int32_t* teacher_ids, const void* teacher_logits, int top,
                        bdr_dtype teacher_dt, float temperature, float* loss, float* lse,
                        float* picked, void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(loss_shape(rows, hidden_size, vocab, rank, dt, top, true));
  LossProblem p = loss_sizes(rows, hidden_size, vocab, rank, dt, top);
  BDR_TRY(loss_markov(p, markov_w1, markov_w2, prev_token));
  BDR_TRY(distill_problem(p, hidden, lm_head_w, teacher_ids, teacher_logits, teacher_dt, temperature));
  return loss_run_forward(p, loss, lse, picked, workspace, workspace_bytes, stream,
                          "dspark_distill_loss launch");
}

int dspark_distill_backward(const void* hidden, int64_t rows, int64_t hidden_size, int64_t vocab,
                            bdr_dtype dt, const void* lm_head_w, const void* markov_w1,
                            const void* markov_w2, int rank, const int32_t* prev_token,
                            const int32_t* teacher_ids, const void* teacher_logits, int top,
                            bdr_dtype teacher_dt, float temperature, const float* lse,
                            const float* picked, const float* loss_grad, void* d_hidden,
                            void* d_lm_head_w, void* d_markov_w1, void* d_markov_w2,
                            void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(loss_shape(rows, hidden_size, vocab, rank, dt, top, true));
  LossProblem p = loss_sizes(rows, hidden_size, vocab, rank, dt, top);
  BDR_TRY(loss_markov(p, markov_w1, markov_w2, prev_token));
  BDR_TRY(distill_problem(p, hidden, lm_head_w, teacher_ids, teacher_logits, teacher_dt, temperature));
  return loss_run_backward(p, LossGrads{d_hidden, d_lm_head_w, d_markov_w1, d_markov_w2}, lse,
                           picked, loss_grad, workspace, workspace_bytes, stream,
                           "dspark_distill_backward launch");
}

// ---------------------------------------------------------------------------- paged attention
namespace {

constexpr int64_t kMaxRequests = int64_t(1) << 20;
constexpr int64_t kMaxContext = int64_t(1) << 30;    // positions of a block table's row
constexpr int64_t kMaxSlotRows = int64_t(1) << 24;
constexpr int64_t kMaxQueryVectors = int64_t(1) << 30;
constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxStride = (int64_t(1) << 30) - 1;   // of a cache, elements: under 2^32 bytes

int table_shape(int64_t batch, int64_t max_pages, int64_t page_size) {
  if (batch < 0) return fail(BDR_EINVAL, "batch must be >= 0");
  if (max_pages < 1) return fail(BDR_EINVAL, "max_pages must be >= 1");
  if (page_size < 1) return fail(BDR_EINVAL, "page_size must be >= 1");
  if (batch > kMaxRequests) return fail(BDR_EUNSUPPORTED, "batch must be <= 2^20");
  if (max_pages > kMaxContext / page_size)
    return fail(BDR_EUNSUPPORTED, "max_pages * page_size must be <= 2^30");
  return BDR_OK;
}

int head_shape(int q_heads, int kv_heads, int head_dim, int dt, bool queries) {
  if (!valid_dtype(dt)) return fail(BDR_EINVAL, "unknown dtype %d", dt);
  if (kv_heads < 1 || q_heads < (queries ? 1 : 0))
    return fail(BDR_EINVAL, "kv_heads must be >= 1 and q_heads >= %d", queries ? 1 : 0);
  if (q_heads > kMaxHeads || kv_heads > kMaxHeads || q_heads + kv_heads > kMaxHeads)
    return fail(BDR_EUNSUPPORTED, "q_heads + kv_heads must be <= %d", kMaxHeads);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(BDR_EUNSUPPORTED, "head_dim %d must be 64, 128 or 256", head_dim);
  return BDR_OK;
}

// elements from the first to the last of [n, heads, dim] at these strides
int64_t head_span(int64_t n, int64_t row, int heads, int64_t head, int dim) {
  return (n - 1) * row + (heads - 1) * head + dim;
}

int head_strides(int64_t rows, int64_t row, int heads, int64_t head, int dt, const char* name) {
  const int e = dt == BDR_BF16 ? 8 : 4;
  if (row < 0 || head < 0 || row % e || head % e)
    return fail(BDR_EINVAL, "the strides of %s must be multiples of %d and >= 0", name, e);
  if ((rows > 0 && row > kMaxElems / rows) || head > kMaxElems / kMaxHeads)
    return fail(BDR_EUNSUPPORTED, "the strides of %s are too large", name);
  return BDR_OK;
}

struct Cache {
  const void *k, *v;
  int64_t pages;
  int page;
  int64_t page_stride, token_stride, head_stride;
  const float *k_scale, *v_scale;
};

int cache_elem(const Cache& c, int dt) { return c.k_scale ? 1 : dt == BDR_BF16 ? 2 : 4; }

int64_t cache_bytes(const Cache& c, int kv_heads, int head_dim, int dt) {
  return ((c.pages - 1) * c.page_stride + (c.page - 1) * c.token_stride +
          (kv_heads - 1) * c.head_stride + head_dim) * cache_elem(c, dt);
}

int cache_shape(const Cache& c, int kv_heads, int dt) {
  if (c.pages < 1) return fail(BDR_EINVAL, "pages must be >= 1");
  if (c.page < 1) return fail(BDR_EINVAL, "page_size must be >= 1");
  if (c.pages > 0x7FFFFFFFLL / c.page)
    return fail(BDR_EUNSUPPORTED, "pages * page_size must be < 2^31");
  if ((c.k_scale == nullptr) != (c.v_scale == nullptr))
    return fail(BDR_EINVAL, "k_scale and v_scale must both be given or both be NULL");
  if (c.k_scale && dt != BDR_BF16) return fail(BDR_EINVAL, "an E4M3 cache goes with bf16 tensors");
  if (c.k_scale) {
    BDR_TRY(need_ptr(c.k_scale, "k_scale", 4));
    BDR_TRY(need_ptr(c.v_scale, "v_scale", 4));
  }
  const int e = 16 / cache_elem(c, dt);
  if (c.page_stride < 0 || c.token_stride < 0 || c.head_stride < 0 || c.page_stride % e ||
      c.token_stride % e || c.head_stride % e)
    return fail(BDR_EINVAL, "the cache's strides must be multiples of 16 bytes and >= 0");
  if (c.page_stride > kMaxStride || c.token_stride > kMaxStride || c.head_stride > kMaxStride)
    return fail(BDR_EUNSUPPORTED, "the cache's strides must be < 2^30 elements");
  // (its bytes stay within 63 bits, so that what overlaps it is seen)
  if (c.pages * c.page_stride > kMaxElems || c.page * c.token_stride > kMaxElems)
    return fail(BDR_EUNSUPPORTED, "the cache must span at most 2^40 elements");
  return BDR_OK;
}

// a written cache's elements lie apart, and its keys apart from its values
int cache_apart(const Cache& c, int kv_heads, int head_dim, int dt) {
  struct Axis {
    int64_t stride, n;
  };
  const int64_t e = cache_elem(c, dt);
  const intptr_t d = static_cast<const char*>(c.v) - static_cast<const char*>(c.k);
  Axis a[4] = {{c.page_stride * e, c.pages}, {c.token_stride * e, c.page},
               {c.head_stride * e, kv_heads}, {d < 0 ? -d : d, 2}};
  std::sort(a, a + 4, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  int64_t reach = head_dim * e;   // bytes that the axes so far span
  for (const Axis& x : a) {
    if (x.n == 1) continue;
    if (x.stride < reach) return fail(BDR_EINVAL, "elements of the cache overlap");
    reach += (x.n - 1) * x.stride;
  }
  return BDR_OK;
}

}  // namespace

int spec_slots(const int32_t* cached, const int32_t* new_tokens, int64_t batch, int64_t max_pages,
               int page_size, int32_t* block_table, const int32_t* page_count,
               int32_t* free_pages, int64_t free_capacity, const int32_t* free_count,
               int64_t max_rows, int32_t* query_offsets, int32_t* kv_len, int32_t* positions,
               int32_t* slots, int32_t* page_count_out, int32_t* free_count_out, int32_t* status,
               void* stream) {
  BDR_TRY(table_shape(batch, max_pages, page_size));
  if (free_capacity < 0) return fail(BDR_EINVAL, "free_capacity must be >= 0");
  if (free_capacity > 0x7FFFFFFFLL) return fail(BDR_EUNSUPPORTED, "free_capacity must be < 2^31");
  if (max_rows < 0) return fail(BDR_EINVAL, "max_rows must be >= 0");
  if (max_rows > kMaxSlotRows) return fail(BDR_EUNSUPPORTED, "max_rows must be <= 2^24");
  if (batch > 0) {
    BDR_TRY(need_ptr(cached, "cached", 4));
    BDR_TRY(need_ptr(new_tokens, "new_tokens", 4));
    BDR_TRY(need_ptr(block_table, "block_table", 4));
    BDR_TRY(need_ptr(page_count, "page_count", 4));
    BDR_TRY(need_ptr(kv_len, "kv_len", 4));
    BDR_TRY(need_ptr(page_count_out, "page_count_out", 4));
  }
  if (free_capacity > 0) BDR_TRY(need_ptr(free_pages, "free_pages", 4));
  BDR_TRY(need_ptr(free_count, "free_count", 4));
  BDR_TRY(need_ptr(query_offsets, "query_offsets", 4));
  if (max_rows > 0) {
    BDR_TRY(need_ptr(positions, "positions", 4));
    BDR_TRY(need_ptr(slots, "slots", 4));
  }
  BDR_TRY(need_ptr(free_count_out, "free_count_out", 4));
  BDR_TRY(need_ptr(status, "status", 4));
  auto given = [](const void* p, int64_t n) { return n > 0 ? p : nullptr; };
  const Span in_count{given(page_count, batch), batch * 4, "page_count"};
  const Span in_free{free_count, 4, "free_count"};
  const Span out_count{given(page_count_out, batch), batch * 4, "page_count_out"};
  const Span out_free{free_count_out, 4, "free_count_out"};
  const std::initializer_list<Span> outs = {
      {given(block_table, batch), batch * max_pages * 4, "block_table"},
      {given(free_pages, free_capacity), free_capacity * 4, "free_pages"},
      {query_offsets, (batch + 1) * 4, "query_offsets"},
      {given(kv_len, batch), batch * 4, "kv_len"},
      {given(positions, max_rows), max_rows * 4, "positions"},
      {given(slots, max_rows), max_rows * 4, "slots"},
      {status, 4, "status"}};
  const Span in_cached{given(cached, batch), batch * 4, "cached"};
  const Span in_new{given(new_tokens, batch), batch * 4, "new_tokens"};
  BDR_TRY(no_overlap(outs, {in_cached, in_new, in_count, in_free, out_count, out_free}));
  BDR_TRY(no_overlap({out_count, out_free}, {in_cached, in_new}));
  if (page_count_out != page_count) BDR_TRY(no_overlap({out_count}, {in_count}));
  if (free_count_out != free_count) BDR_TRY(no_overlap({out_free}, {in_free}));
  BDR_TRY(no_overlap({out_count}, {in_free}));
  BDR_TRY(no_overlap({out_free}, {in_count}));
  BDR_TRY(check_device());
  const SlotProblem p{cached, new_tokens, static_cast<int32_t>(batch), static_cast<int32_t>(max_pages),
                      page_size, static_cast<int32_t>(free_capacity), static_cast<int32_t>(max_rows),
                      block_table, page_count, free_pages, free_count, query_offsets, kv_len, positions,
                      slots, page_count_out, free_count_out, status};
  const hipError_t e = launch_slots(p, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "spec_slots launch");
  return BDR_OK;
}

int dspark_qk_norm_rope(const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k,
                        int64_t k_row_stride, int64_t k_head_stride, const void* v,
                        int64_t v_row_stride, int64_t v_head_stride, int64_t rows, int q_heads,
                        int kv_heads, int head_dim, bdr_dtype dt, const int32_t* positions,
                        const float* inv_freq, int rot_dim, int interleaved, const void* q_weight,
                        const void* k_weight, float eps, void* q_out, void* k_out,
                        const int32_t* slots, void* k_cache, void* v_cache, int64_t pages,
                        int page_size, int64_t page_stride, int64_t token_stride,
                        int64_t head_stride, const float* k_scale, const float* v_scale,
                        void* stream) {
  BDR_TRY(head_shape(q_heads, kv_heads, head_dim, dt, false));
  if (rows < 0) return fail(BDR_EINVAL, "rows must be >= 0");
  if (rows >= kMaxSlotRows) return fail(BDR_EUNSUPPORTED, "rows must be < 2^24");
  if (rot_dim < 16 || rot_dim > head_dim || rot_dim % 16)
    return fail(BDR_EINVAL, "rot_dim %d must be a multiple of 16 in 16 .. head_dim", rot_dim);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(BDR_EINVAL, "eps must be finite and >= 0");
  if (q_heads == 0 && k_weight) q_weight = k_weight;   // (there is nothing that would read it)
  if ((q_weight == nullptr) != (k_weight == nullptr))
    return fail(BDR_EINVAL, "q_weight and k_weight must both be given or both be NULL");
  if ((k_cache == nullptr) != (v_cache == nullptr))
    return fail(BDR_EINVAL, "k_cache and v_cache must both be given or both be NULL");
  const bool cached = k_cache != nullptr;
  const Cache c{k_cache, v_cache, pages, page_size, page_stride, token_stride, head_stride, k_scale, v_scale};
  if (cached) {
    BDR_TRY(need_ptr(k_cache, "k_cache"));
    BDR_TRY(need_ptr(v_cache, "v_cache"));
    BDR_TRY(cache_shape(c, kv_heads, dt));
    BDR_TRY(cache_apart(c, kv_heads, head_dim, dt));
  } else if (k_scale || v_scale) {
    return fail(BDR_EINVAL, "scales are given without a cache");
  }
  BDR_TRY(head_strides(rows, q_row_stride, q_heads, q_head_stride, dt, "q"));
  BDR_TRY(head_strides(rows, k_row_stride, kv_heads, k_head_stride, dt, "k"));
  BDR_TRY(head_strides(rows, v_row_stride, kv_heads, v_head_stride, dt, "v"));
  if (rows == 0) return BDR_OK;
  if (q_heads) {
    BDR_TRY(need_ptr(q, "q"));
    BDR_TRY(need_ptr(q_out, "q_out"));
  }
  BDR_TRY(need_ptr(k, "k"));
  if (k_out) BDR_TRY(need_ptr(k_out, "k_out"));
  if (cached) {
    BDR_TRY(need_ptr(v, "v"));
    BDR_TRY(need_ptr(slots, "slots", 4));
  } else if (!k_out) {
    return fail(BDR_EINVAL, "keys go nowhere: k_out or a cache is needed");
  }
  BDR_TRY(need_ptr(positions, "positions", 4));
  BDR_TRY(need_ptr(inv_freq, "inv_freq", 4));
  if (q_weight) {
    BDR_TRY(need_ptr(k_weight, "k_weight"));
    BDR_TRY(need_ptr(q_weight, "q_weight"));
  }
  const int64_t es = dt == BDR_BF16 ? 2 : 4;
  const Span sq{q_heads ? q : nullptr, q_heads ? head_span(rows, q_row_stride, q_heads, q_head_stride, head_dim) * es : 0, "q"};
  const Span sk{k, head_span(rows, k_row_stride, kv_heads, k_head_stride, head_dim) * es, "k"};
  const Span sv{cached ? v : nullptr, head_span(rows, v_row_stride, kv_heads, v_head_stride, head_dim) * es, "v"};
  const Span oq{q_heads ? q_out : nullptr, rows * q_heads * head_dim * es, "q_out"};
  const Span ok{k_out, rows * kv_heads * head_dim * es, "k_out"};
  const int64_t cb = cached ? cache_bytes(c, kv_heads, head_dim, dt) : 0;
  const Span ck{k_cache, cb, "k_cache"}, cv{v_cache, cb, "v_cache"};
  const std::initializer_list<Span> rest = {{positions, rows * 4, "positions"},
                                            {inv_freq, rot_dim * 2, "inv_freq"},
                                            {k_weight, head_dim * es, "k_weight"},
                                            {q_weight, head_dim * es, "q_weight"},
                                            {cached ? slots : nullptr, rows * 4, "slots"},
                                            {k_scale, kv_heads * 4, "k_scale"},
                                            {v_scale, kv_heads * 4, "v_scale"}};
  BDR_TRY(no_overlap({oq, ok}, rest));
  BDR_TRY(no_overlap({ck}, rest));
  BDR_TRY(no_overlap({cv}, rest));
  BDR_TRY(no_overlap({ck}, {sq, sk, sv, oq, ok}));   // (keys and values may interleave)
  BDR_TRY(no_overlap({cv}, {sq, sk, sv, oq, ok}));
  auto in_place = [&](const void* in, const void* out, int64_t row, int64_t head, int heads) {
    // contiguous (the stride of an axis of one entry says nothing)
    return in == out && (heads == 1 || head == head_dim) &&
           (rows == 1 || row == static_cast<int64_t>(heads) * head_dim);
  };
  if (!(q_heads && in_place(q, q_out, q_row_stride, q_head_stride, q_heads))) BDR_TRY(no_overlap({oq}, {sq}));
  if (!(k_out && in_place(k, k_out, k_row_stride, k_head_stride, kv_heads))) BDR_TRY(no_overlap({ok}, {sk}));
  BDR_TRY(no_overlap({oq}, {sk, sv}));
  BDR_TRY(no_overlap({ok}, {sq, sv}));
  BDR_TRY(check_device());
  QkProblem p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.k_row = k_row_stride;
  p.k_head = k_head_stride;
  p.v_row = v_row_stride;
  p.v_head = v_head_stride;
  p.rows = rows;
  p.hq = q_heads;
  p.hkv = kv_heads;
  p.dim = head_dim;
  p.half = rot_dim / 2;
  p.interleaved = interleaved != 0;
  p.fp8 = k_scale != nullptr;
  p.dt = dt;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.wq = q_weight;
  p.wk = k_weight;
  p.eps = eps;
  p.q_out = q_out;
  p.k_out = k_out;
  p.slots = slots;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.page = cached ? page_size : 1;
  p.slots_held = cached ? static_cast<int32_t>(pages * page_size) : 0;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  const hipError_t e = launch_qk(p, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dspark_qk_norm_rope launch");
  return BDR_OK;
}

namespace {

int attn_shape(int64_t rows, int q_heads, int kv_heads, int head_dim, int dt, int64_t batch,
               int64_t max_pages, int64_t page_size) {
  BDR_TRY(head_shape(q_heads, kv_heads, head_dim, dt, true));
  if (q_heads % kv_heads)
    return fail(BDR_EINVAL, "q_heads %d must be a multiple of kv_heads %d", q_heads, kv_heads);
  if (rows < 0) return fail(BDR_EINVAL, "rows must be >= 0");
  if (rows > kMaxQueryVectors / q_heads)
    return fail(BDR_EUNSUPPORTED, "rows * q_heads must be <= 2^30");
  return table_shape(batch, max_pages, page_size);
}

AttnProblem attn_sizes(int64_t rows, int q_heads, int kv_heads, int head_dim, bdr_dtype dt,
                       int64_t batch, int64_t max_pages, int page_size) {
  AttnProblem p{};
  p.rows = rows;
  p.hq = q_heads;
  p.hkv = kv_heads;
  p.group = q_heads / kv_heads;
  p.dim = head_dim;
  p.dt = dt;
  p.batch = static_cast<int>(batch);
  p.width = static_cast<int>(max_pages);
  p.page = page_size;
  return p;
}

}  // namespace

size_t dflash_paged_attention_workspace_bytes(int64_t rows, int q_heads, int kv_heads, int head_dim,
                                              bdr_dtype dt, int64_t batch, int64_t max_pages,
                                              int page_size) {
  if (attn_shape(rows, q_heads, kv_heads, head_dim, dt, batch, max_pages, page_size) != BDR_OK ||
      rows == 0 || batch == 0)
    return 0;
  return attn_workspace(attn_sizes(rows, q_heads, kv_heads, head_dim, dt, batch, max_pages, page_size));
}

int dflash_paged_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride, int64_t rows,
                           int q_heads, int kv_heads, int head_dim, bdr_dtype dt,
                           const void* k_cache, const void* v_cache, int64_t pages, int page_size,
                           int64_t page_stride, int64_t token_stride, int64_t head_stride,
                           const float* k_scale, const float* v_scale, const int32_t* block_table,
                           int64_t batch, int64_t max_pages, const int32_t* query_offsets,
                           const int32_t* kv_len, float scale, int causal, int window, void* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  BDR_TRY(attn_shape(rows, q_heads, kv_heads, head_dim, dt, batch, max_pages, page_size));
  const Cache c{k_cache, v_cache, pages, page_size, page_stride, token_stride, head_stride, k_scale, v_scale};
  BDR_TRY(cache_shape(c, kv_heads, dt));
  BDR_TRY(head_strides(rows, q_row_stride, q_heads, q_head_stride, dt, "q"));
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(BDR_EINVAL, "scale must be finite and > 0");
  if (window < 0) return fail(BDR_EINVAL, "window must be >= 0");
  if (rows == 0 || batch == 0) return BDR_OK;
  BDR_TRY(need_ptr(q, "q"));
  BDR_TRY(need_ptr(k_cache, "k_cache"));
  BDR_TRY(need_ptr(v_cache, "v_cache"));
  BDR_TRY(need_ptr(block_table, "block_table", 4));
  BDR_TRY(need_ptr(query_offsets, "query_offsets", 4));
  BDR_TRY(need_ptr(kv_len, "kv_len", 4));
  BDR_TRY(need_ptr(out, "out"));
  if (lse) BDR_TRY(need_ptr(lse, "lse", 4));
  AttnProblem p = attn_sizes(rows, q_heads, kv_heads, head_dim, dt, batch, max_pages, page_size);
  const size_t need = attn_workspace(p);
  BDR_TRY(need_ws(workspace, workspace_bytes, need));
  const int64_t es = dt == BDR_BF16 ? 2 : 4;
  const int64_t cb = cache_bytes(c, kv_heads, head_dim, dt);
  BDR_TRY(no_overlap({{out, rows * q_heads * head_dim * es, "out"},
                      {lse, rows * q_heads * 4, "lse"},
                      {need ? workspace : nullptr, static_cast<int64_t>(need), "workspace"}},
                     {{q, head_span(rows, q_row_stride, q_heads, q_head_stride, head_dim) * es, "q"},
                      {k_cache, cb, "k_cache"},
                      {v_cache, cb, "v_cache"},
                      {k_scale, kv_heads * 4, "k_scale"},
                      {v_scale, kv_heads * 4, "v_scale"},
                      {block_table, batch * max_pages * 4, "block_table"},
                      {query_offsets, (batch + 1) * 4, "query_offsets"},
                      {kv_len, batch * 4, "kv_len"}}));
  BDR_TRY(check_device());
  p.q = q;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.fp8 = k_scale != nullptr;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.pages = static_cast<int>(pages);
  const int64_t ce = cache_elem(c, dt);
  p.page_bytes = static_cast<uint32_t>(page_stride * ce);
  p.token_bytes = static_cast<uint32_t>(token_stride * ce);
  p.head_bytes = head_stride * ce;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = block_table;
  p.offsets = query_offsets;
  p.kv_len = kv_len;
  p.scale = scale;
  p.causal = causal != 0;
  // a window past every context is none
  p.window = window >= max_pages * page_size ? 0 : window;
  p.out = out;
  p.lse = lse;
  const hipError_t e = launch_attn(p, workspace, as_stream(stream));
  if (e != hipSuccess) return hip_fail(e, "dflash_paged_attention launch");
  return BDR_OK;
}

}  // extern "C"
