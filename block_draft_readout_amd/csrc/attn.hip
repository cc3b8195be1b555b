// Host side of the attention over a paged cache: which variant, how many
// workgroups, and the workspace of its partials.

#include <algorithm>
#include <limits>

#include "attn_run.h"

namespace bdr {

namespace {

constexpr int64_t kCus = 256;                    // compute units of an MI355X
constexpr int64_t kMaxGrid = int64_t(1) << 20;   // workgroups

struct Choice {
  int few;            // 16-row tiles of a few-row variant; 0, -1: many rows in tiles of 128, 256
  int bm;             // rows of a row tile
  int64_t shares, min_share;
  int whole;
};

// Measured: 16 requests' tokens over 8192 bf16 keys, 40 query and 8 kv heads of 128, pages of 16,
// unless said otherwise; one kind of kernel against the next.
//
// Few rows, each wave with all of them and keys of its own, up to 64 packed rows (40 rows 107
// against 120 us, 50 rows 112 against 121; at 80 they no longer fit the registers): what bounds
// them is the cache's bytes.  Wider rows hold fewer (D = 256: 32 rows 65 against 68 us; fp32 of 256:
// none, four waves' tiles are more than LDS holds).
// Row tiles of 128, keys shared by four waves, up to 128 rows (65 rows 120 against 163 us, 80 rows
// 125 against 176: a tile of 256 would be empty for the most part).
// Row tiles of 256, two waves of a SIMD in opposite phases, past that (130 rows 177 against 183 us,
// 200 rows 185 against 198, 520 rows 482 against 557); built where their registers and LDS suffice.
// A last tile that is mostly empty costs a whole one: 260 rows 265 us, 520 rows 461.
//
// The rows are those of a request on average, and the measured requests are alike: the lengths are
// on the device.  A call whose requests differ much is best made in two: a chunk of 2048 tokens
// over 8192 keys (4 query heads a kv head) takes 267 us, 31 single tokens over 2000 to 8000 keys
// 115, both together 427; with 255 single tokens, whose kernel the chunk then shares, 1561 against
// 267 + 846.
Choice choose(const AttnProblem& p) {
  Choice c{};
  // rows of a request and kv head on average
  const int64_t rows = (p.rows * p.group + p.batch - 1) / p.batch;
  const int most = p.dt == BDR_F32 ? (p.dim == 256 ? 0 : 2) : p.dim == 256 ? 2 : 4;
  c.few = rows <= 16 * most ? static_cast<int>((rows + 15) / 16) : 0;
  if (c.few == 0 && rows > 128 && p.dt == BDR_BF16 && (p.dim == 128 || (p.dim == 64 && !p.fp8))) c.few = -1;
  c.bm = c.few > 0 ? 16 * c.few : c.few == 0 ? 128 : 256;
  const int64_t longest = static_cast<int64_t>(p.width) * p.page;
  const int64_t tiles = (p.rows * p.group + c.bm - 1) / c.bm + p.batch;   // row tiles at most
  const int elem = p.fp8 ? 1 : p.dt == BDR_F32 ? 4 : 2;
  // One launch instead of two where the longest table is through in a few rounds of a workgroup's
  // waves.  A token over 100 keys 8.2 against 11.3 us, over 1000 the same, over 2000 23 against 13.7;
  // 4 x 100 tokens over 200 keys 21 against 58 us, 8 prompts of 128 18 against 60; fp32, 5 x 7
  // tokens over 128 keys 11 against 28 us, over 512 19 against 24, over 1001 29 against 25.  It is
  // the table's width that is known here: contexts as short in a wide table take the longer times.
  // Every workgroup looks through the lengths of all requests: 1000 tokens over up to 1024 keys 628
  // against 405 us.
  const int64_t at_once = c.few > 0 ? 128 * few_waves(elem, p.dim) : 256;
  c.whole = longest <= at_once && tiles * p.hkv <= kMaxGrid;
  // else as many shares as the chip holds at once
  c.shares = c.whole ? tiles : std::max<int64_t>(1, attn_per_cu(c.few, elem, p.dim) * kCus / p.hkv);
  // key tiles that are worth a workgroup and its partials (8 tokens over 4096 keys, one request: 19
  // us, with 2 tiles 26, with 24 tiles 25; 4 x 100 tokens over 2048 keys 47.5, 48 and 82 us)
  c.min_share = 8;
  return c;
}

}  // namespace

static size_t workspace_of(const AttnProblem& p) {
  const Choice c = choose(p);
  if (c.whole) return 0;
  const size_t slots = 2 * static_cast<size_t>(c.shares) * p.hkv * c.bm;
  return align256(slots * p.dim * sizeof(float)) + align256(slots * sizeof(float2)) +
         align256(static_cast<size_t>(c.shares) * p.hkv * kRecord * sizeof(int32_t));
}

// (whatever the cache holds: its type is not among the sizes that are asked for)
size_t attn_workspace(const AttnProblem& p) {
  AttnProblem a = p, b = p;
  a.fp8 = 0;
  b.fp8 = 1;
  return std::max(workspace_of(a), workspace_of(b));
}

hipError_t launch_attn(const AttnProblem& p, void* workspace, hipStream_t stream) {
  const Choice c = choose(p);
  AttnArgs g{};
  g.p = p;
  g.shares = c.shares;
  g.min_share = c.min_share;
  g.whole = c.whole;
  g.scale2 = std::min(p.scale * kLog2e, std::numeric_limits<float>::max());
  // s = ceil(log2 page), magic = ceil(2^(31 + s) / page): exact for keys below 2^31
  while ((int64_t(1) << g.page_shift) < p.page) ++g.page_shift;
  g.page_magic = static_cast<uint32_t>(((uint64_t(1) << (31 + g.page_shift)) + p.page - 1) / p.page);
  if (!c.whole) {
    const size_t slots = 2 * static_cast<size_t>(c.shares) * p.hkv * c.bm;
    char* at = static_cast<char*>(workspace);
    g.part_o = reinterpret_cast<float*>(at);
    at += align256(slots * p.dim * sizeof(float));
    g.part_ml = reinterpret_cast<float2*>(at);
    at += align256(slots * sizeof(float2));
    g.record = reinterpret_cast<int32_t*>(at);
  }
  if (p.dt == BDR_F32) return launch_attn_f32(g, c.few, stream);
  return p.fp8 ? launch_attn_fp8(g, c.few, stream) : launch_attn_bf16(g, c.few, stream);
}

}  // namespace bdr
