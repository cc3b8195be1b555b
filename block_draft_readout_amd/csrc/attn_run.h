// Launch of one attention variant, shared by the attention's translation units.
#pragma once

#include "attn.h"

namespace bdr {

// which: 0 few rows, 1 some rows, 2 many rows
hipError_t launch_attn_bf16(const AttnArgs& g, int which, hipStream_t stream);
hipError_t launch_attn_fp8(const AttnArgs& g, int which, hipStream_t stream);
hipError_t launch_attn_f32(const AttnArgs& g, int which, hipStream_t stream);

template <typename T>
hipError_t run_attn(const AttnArgs& g, hipStream_t stream) {
  const int64_t grid = (g.slabs + 7) / 8 * 8;
  hipLaunchKernelGGL((attn_kernel<T>), dim3(static_cast<uint32_t>(grid)), dim3(T::THREADS), 0, stream, g);
  if (!g.whole && g.slabs > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_join_kernel<T>), dim3(static_cast<uint32_t>(g.slabs - 1), 4), dim3(256), 0,
                       stream, g);
  }
  return hipGetLastError();
}

}  // namespace bdr
