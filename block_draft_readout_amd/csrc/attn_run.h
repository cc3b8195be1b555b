// Launch of one attention variant, shared by the attention's translation units.
#pragma once

#include "attn.h"

namespace bdr {

// few: 16-row tiles of a few-row variant, 0 or -1: many rows, in row tiles of 128 or 256
hipError_t launch_attn_bf16(const AttnArgs& g, int few, hipStream_t stream);
hipError_t launch_attn_fp8(const AttnArgs& g, int few, hipStream_t stream);
hipError_t launch_attn_f32(const AttnArgs& g, int few, hipStream_t stream);

template <typename T>
hipError_t run_attn(const AttnArgs& g, hipStream_t stream) {
  const uint32_t grid = static_cast<uint32_t>(g.shares * g.p.hkv);
  hipLaunchKernelGGL((attn_kernel<T>), dim3(grid), dim3(T::THREADS), 0, stream, g);
  if (!g.whole && g.shares > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // row blocks: most workgroups find nothing to join, so no more than tall tiles need
    constexpr int blocks = std::min(8, T::BM * (T::D / 4) / 256);
    hipLaunchKernelGGL((attn_join_kernel<T>), dim3(grid - g.p.hkv, blocks), dim3(256), 0, stream, g);
  }
  return hipGetLastError();
}

// the built variants of a head size
template <typename C, typename S, int D, int KT, int FEW, bool TALL>
hipError_t run_attn_dim(const AttnArgs& g, int few, hipStream_t stream) {
  switch (few) {
    case 1: return run_attn<AttnFew<C, S, D, 1>>(g, stream);
    case 2: return run_attn<AttnFew<C, S, D, 2>>(g, stream);
    case 3: if constexpr (FEW >= 3) return run_attn<AttnFew<C, S, D, 3>>(g, stream); break;
    case 4: if constexpr (FEW >= 4) return run_attn<AttnFew<C, S, D, 4>>(g, stream); break;
    case -1: if constexpr (TALL) return run_attn<AttnTall<C, S, D, KT>>(g, stream); break;
    default: return run_attn<AttnMany<C, S, D, 4, 1, KT>>(g, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace bdr
