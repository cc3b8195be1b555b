// Attention over a paged e4m3 cache, queries and output in bf16.
#include "attn_run.h"

namespace bdr {

template <int D, int KT>
static hipError_t run(const AttnArgs& g, int which, hipStream_t stream) {
  if (which == 0) return run_attn<AttnTile<uint8_t, uint16_t, D, 1, 4, 1, 32>>(g, stream);
  if constexpr (D <= 128)
    if (which == 1) return run_attn<AttnTile<uint8_t, uint16_t, D, 1, 4, 2, 32>>(g, stream);
  return run_attn<AttnTile<uint8_t, uint16_t, D, 4, 1, 1, KT>>(g, stream);
}

hipError_t launch_attn_fp8(const AttnArgs& g, int which, hipStream_t stream) {
  switch (g.p.dim) {
    case 64: return run<64, 64>(g, which, stream);
    case 128: return run<128, 64>(g, which, stream);
    default: return run<256, 32>(g, which, stream);
  }
}

}  // namespace bdr
