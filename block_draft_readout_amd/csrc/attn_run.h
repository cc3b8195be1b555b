// Launch of one attention variant, shared by the attention's translation units.
#pragma once

#include "attn.h"

namespace bdr {

// few: 16-row tiles of a few-row variant, 0 or -1: many rows, in row tiles of 128 or 256
hipError_t launch_attn_bf16(const AttnArgs& g, int few, hipStream_t stream);
hipError_t launch_attn_fp8(const AttnArgs& g, int few, hipStream_t stream);
hipError_t launch_attn_f32(const AttnArgs& g, int few, hipStream_t stream);

// Workgroups that a compute unit holds of a variant that shares row tiles (few as below).
constexpr int attn_per_cu(int few, int cache_elem, int dim) {
  if (few < 0) return 1;
  if (few == 0) return cache_elem * dim <= 256 && dim <= 128 ? 2 : 1;
  return dim * few <= (cache_elem == 1 ? 256 : 384) && cache_elem * dim <= 256 && dim <= 128 ? 2 : 1;
}

// waves of a few-row workgroup that takes whole row tiles: 16 KB of LDS each
constexpr int few_waves(size_t cache_elem, int dim) {
  return cache_elem == 1 ? (dim <= 128 ? 8 : 4) : cache_elem * dim <= 256 ? 8 : 4;
}

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

// Few rows.  Where a row tile is one workgroup's, eight waves walk its keys if their tiles fit LDS.
template <typename C, typename S, int D, int RT>
hipError_t run_attn_few(const AttnArgs& g, hipStream_t stream) {
  if constexpr (few_waves(sizeof(C), D) == 8)
    if (g.whole) return run_attn<AttnFew<C, S, D, RT, 8>>(g, stream);
  return run_attn<AttnFew<C, S, D, RT, 4>>(g, stream);
}

// the built variants of a head size
template <typename C, typename S, int D, int KT, int FEW, bool TALL>
hipError_t run_attn_dim(const AttnArgs& g, int few, hipStream_t stream) {
  switch (few) {
    case 1: return run_attn_few<C, S, D, 1>(g, stream);
    case 2: return run_attn_few<C, S, D, 2>(g, stream);
    case 3: if constexpr (FEW >= 3) return run_attn_few<C, S, D, 3>(g, stream); break;
    case 4: if constexpr (FEW >= 4) return run_attn_few<C, S, D, 4>(g, stream); break;
    case -1: if constexpr (TALL) return run_attn<AttnTall<C, S, D, KT>>(g, stream); break;
    default: return run_attn<AttnMany<C, S, D, 4, KT>>(g, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace bdr
