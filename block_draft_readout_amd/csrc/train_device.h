// Device-side helpers shared by the training kernels (row norm, losses).
#pragma once

#include "gemm_kernels.h"

namespace bdr {

// two floats -> bfloat16 bits (a in the low half), round to nearest even with
// the hardware conversion: infinities and NaN stay what they are
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2_t{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// v rounded to the storage type
template <typename S> __device__ __forceinline__ S rounded(float v);
template <> __device__ __forceinline__ float rounded<float>(float v) { return v; }
template <> __device__ __forceinline__ uint16_t rounded<uint16_t>(float v) {
  return static_cast<uint16_t>(pack_bf16(v, 0.f));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

}  // namespace bdr
