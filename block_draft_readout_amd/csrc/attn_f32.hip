// Attention over a paged fp32 cache.
#include "attn_run.h"

namespace bdr {

hipError_t launch_attn_f32(const AttnArgs& g, int few, hipStream_t stream) {
  switch (g.p.dim) {
    case 64: return run_attn_dim<float, float, 64, 32, 2, false>(g, few, stream);
    case 128: return run_attn_dim<float, float, 128, 32, 2, false>(g, few, stream);
    default: return run_attn<AttnMany<float, float, 256, 4, 32>>(g, stream);
  }
}

}  // namespace bdr
