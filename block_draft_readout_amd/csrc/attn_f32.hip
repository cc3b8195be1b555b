// Attention over a paged fp32 cache.
#include "attn_run.h"

namespace bdr {

template <int D>
static hipError_t run(const AttnArgs& g, int which, hipStream_t stream) {
  if constexpr (D <= 128)
    if (which == 0) return run_attn<AttnTile<float, float, D, 1, 4, 1, 32>>(g, stream);
  return run_attn<AttnTile<float, float, D, 4, 1, 1, 32>>(g, stream);
}

hipError_t launch_attn_f32(const AttnArgs& g, int which, hipStream_t stream) {
  switch (g.p.dim) {
    case 64: return run<64>(g, which, stream);
    case 128: return run<128>(g, which, stream);
    default: return run<256>(g, which, stream);
  }
}

}  // namespace bdr
