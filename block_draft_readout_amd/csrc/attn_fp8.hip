// Attention over a paged e4m3 cache, queries and output in bf16.
#include "attn_run.h"

namespace bdr {

hipError_t launch_attn_fp8(const AttnArgs& g, int few, hipStream_t stream) {
  switch (g.p.dim) {
    case 64: return run_attn_dim<uint8_t, uint16_t, 64, 64, 4, false>(g, few, stream);
    case 128: return run_attn_dim<uint8_t, uint16_t, 128, 64, 4, true>(g, few, stream);
    default: return run_attn_dim<uint8_t, uint16_t, 256, 32, 2, false>(g, few, stream);
  }
}

}  // namespace bdr
