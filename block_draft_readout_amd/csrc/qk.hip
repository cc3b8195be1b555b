// Norm of queries and keys for each head, rotation by position and the write of
// keys and values into the paged cache (gfx950).
//
//   y = x (sum x^2 / D + eps)^-1/2 w                  (each head; no w: y = x)
//   (y1, y2) -> (y1 cos a - y2 sin a, y2 cos a + y1 sin a),  a = position inv_freq[i]
// for the pairs i < half; the features from 2 half on stay.  Keys go to their
// token's slot of the cache, values beside them, either in the tensors' type or
// as e4m3(y / scale of the head).
//
// A few flops per byte: HBM bounds it, so one pass reads q, k and v and writes q
// and the cache.  A vector is held by D / 16 lanes; each lane holds the two
// chunks of 8 features that the rotation pairs (interleaved pairs lie inside a
// chunk), so the only exchange between lanes is the sum of squares.  The angles
// of a token are the same for all of its heads: the workgroup computes them once
// into LDS, under the loads of the first vectors.
//
// Angles are products in 64 bits, reduced by quarter turns there: a position of
// 2^20 would leave 2^-4 of an fp32 angle.  Sine and cosine of the rest, at most
// pi / 4, are their Taylor sums in 64 bits too (the first term left out is under
// 2e-10) and rounded once: in fp32 they cost an ulp more and no time less (8192
// tokens of 40 + 2 x 8 heads 50.7 against 50.9 us).  Sums of squares, products and
// quotients are fp32; what is stored is rounded once.

#include <algorithm>

#include "bdr_internal.h"
#include "train_device.h"

namespace bdr {

constexpr int kQkThreads = 256;

__device__ __forceinline__ float2 turn_of(int32_t position, float inv_freq) {
  const double t = static_cast<double>(position) * static_cast<double>(inv_freq) * 0.63661977236758134308;
  const double q = rint(t);   // quarter turns
  const double f = (t - q) * 1.57079632679489661923;
  const double f2 = f * f;
  double s = -2.5052108385441719e-8;
  s = fma(s, f2, 2.7557319223985891e-6);
  s = fma(s, f2, -1.9841269841269841e-4);
  s = fma(s, f2, 8.3333333333333333e-3);
  s = fma(s, f2, -1.6666666666666667e-1);
  s = fma(s * f2, f, f);
  double c = -2.7557319223985888e-7;
  c = fma(c, f2, 2.4801587301587302e-5);
  c = fma(c, f2, -1.3888888888888889e-3);
  c = fma(c, f2, 4.1666666666666667e-2);
  c = fma(c, f2, -0.5);
  c = fma(c, f2, 1.0);
  const int k = static_cast<int>(static_cast<int64_t>(q) & 3);
  const float cs = static_cast<float>(k & 1 ? s : c), sn = static_cast<float>(k & 1 ? c : s);
  return float2{k == 1 || k == 2 ? -cs : cs, k >= 2 ? -sn : sn};
}

// 8 features as fp32, from and to the tensors' type
template <typename S>
__device__ __forceinline__ void load8(const S* p, float (&f)[8]) {
  if constexpr (sizeof(S) == 2) {
    const u32x4_t v = load16(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(v[e] << 16);
      f[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
    }
  } else {
    const u32x4_t a = load16(p), b = load16(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = __uint_as_float(a[e]);
      f[4 + e] = __uint_as_float(b[e]);
    }
  }
}

template <typename S>
__device__ __forceinline__ void store8(S* p, const float (&f)[8]) {
  if constexpr (sizeof(S) == 2) {
    *reinterpret_cast<u32x4_t*>(p) = u32x4_t{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                             pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  } else {
    *reinterpret_cast<f32x4_t*>(p) = f32x4_t{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{f[4], f[5], f[6], f[7]};
  }
}

// e4m3 codes of f / scale: values past the largest go to it, NaN stays NaN
__device__ __forceinline__ void store8(uint8_t* p, const float (&f)[8], float scale) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = f[e] / scale;
    x[e] = x[e] > 448.f ? 448.f : x[e];
    x[e] = x[e] < -448.f ? -448.f : x[e];
  }
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], b, true);
  *reinterpret_cast<int2*>(p) = int2{a, b};
}

// TOKENS tokens per workgroup, each with kQkThreads / TOKENS threads
template <typename S, int D, bool FP8, int TOKENS>
__global__ __launch_bounds__(kQkThreads) void qk_kernel(const QkProblem g) {
  constexpr int LV = D / 16;                       // lanes of a vector
  constexpr int SLOTS = kQkThreads / TOKENS / LV;  // vectors at a time
  __shared__ float2 turn[TOKENS][D / 2];
  const int tid = static_cast<int>(threadIdx.x);
  const int tok = tid / (kQkThreads / TOKENS);
  const int in = tid % (kQkThreads / TOKENS);
  const int lane = in % LV;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * TOKENS + tok;
  const bool live = row < g.rows;
  const int64_t r = live ? row : 0;
  const int half = g.half;
  // this lane's two chunks: features i and half + i of the rotated part, or neighbours
  const int turned = half / 8;   // chunks of each half
  int c0, c1;
  if (g.interleaved || lane >= turned) {
    c0 = 2 * lane;
    c1 = c0 + 1;
  } else {
    c0 = lane;
    c1 = lane + turned;
  }
  const int heads = g.hq + g.hkv;
  const int vectors = heads + (g.k_cache ? g.hkv : 0);
  auto source = [&](int h) -> const S* {
    const S* q = static_cast<const S*>(g.q) + r * g.q_row + static_cast<int64_t>(h) * g.q_head;
    const S* k = static_cast<const S*>(g.k) + r * g.k_row + static_cast<int64_t>(h - g.hq) * g.k_head;
    const S* v = static_cast<const S*>(g.v) + r * g.v_row + static_cast<int64_t>(h - heads) * g.v_head;
    return h < g.hq ? q : h < heads ? k : v;
  };
  float f[2][8], w[2][2][8];
  int h = in / LV;
  if (h < vectors) {
    const S* p = source(h);
    load8(p + 8 * c0, f[0]);
    load8(p + 8 * c1, f[1]);
  }
  if (g.wq) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const S* wv = static_cast<const S*>(k ? g.wk : g.wq);
      load8(wv + 8 * c0, w[k][0]);
      load8(wv + 8 * c1, w[k][1]);
    }
  }
  for (int i = tid; i < TOKENS * half; i += kQkThreads) {
    const int t = i / half;
    const int64_t rt = min(static_cast<int64_t>(blockIdx.x) * TOKENS + t, g.rows - 1);
    turn[t][i - t * half] = turn_of(g.positions[rt], g.inv_freq[i - t * half]);
  }
  int64_t at = -1;
  if (g.k_cache) {
    const int32_t slot = g.slots[r];
    if (slot >= 0 && slot < g.slots_held) {
      const int32_t page = slot / g.page;
      at = page * g.page_stride + (slot - page * g.page) * g.token_stride;
    }
  }
  __syncthreads();
  if (!live) return;
  while (h < vectors) {
    const int next = h + SLOTS;
    float n[2][8];
    if (next < vectors) {
      const S* p = source(next);
      load8(p + 8 * c0, n[0]);
      load8(p + 8 * c1, n[1]);
    }
    if (h < heads) {
      if (g.wq) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += f[0][e] * f[0][e] + f[1][e] * f[1][e];
#pragma unroll
        for (int m = 1; m < LV; m <<= 1) s += __shfl_xor(s, m);
        const float rstd = 1.0f / sqrtf(s * (1.0f / D) + g.eps);
        const bool isk = h >= g.hq;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[0][e] = f[0][e] * rstd * (isk ? w[1][0][e] : w[0][0][e]);
          f[1][e] = f[1][e] * rstd * (isk ? w[1][1][e] : w[0][1][e]);
        }
      }
      if (g.interleaved) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * (k ? c1 : c0) + e;
            if (i < half) {
              const float2 t = turn[tok][i];
              const float x = f[k][2 * e], y = f[k][2 * e + 1];
              f[k][2 * e] = x * t.x - y * t.y;
              f[k][2 * e + 1] = y * t.x + x * t.y;
            }
          }
      } else if (lane < turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 t = turn[tok][8 * lane + e];
          const float x = f[0][e], y = f[1][e];
          f[0][e] = x * t.x - y * t.y;
          f[1][e] = y * t.x + x * t.y;
        }
      }
    }
    if (h < g.hq) {
      S* o = static_cast<S*>(g.q_out) + (row * g.hq + h) * D;
      store8(o + 8 * c0, f[0]);
      store8(o + 8 * c1, f[1]);
    } else {
      const int hk = h < heads ? h - g.hq : h - heads;
      if (h < heads && g.k_out) {
        S* o = static_cast<S*>(g.k_out) + (row * g.hkv + hk) * D;
        store8(o + 8 * c0, f[0]);
        store8(o + 8 * c1, f[1]);
      }
      if (at >= 0) {
        const int64_t to = at + hk * g.head_stride;
        if constexpr (FP8) {
          uint8_t* o = static_cast<uint8_t*>(h < heads ? g.k_cache : g.v_cache) + to;
          const float scale = (h < heads ? g.k_scale : g.v_scale)[hk];
          store8(o + 8 * c0, f[0], scale);
          store8(o + 8 * c1, f[1], scale);
        } else {
          S* o = static_cast<S*>(h < heads ? g.k_cache : g.v_cache) + to;
          store8(o + 8 * c0, f[0]);
          store8(o + 8 * c1, f[1]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[0][e] = n[0][e];
      f[1][e] = n[1][e];
    }
    h = next;
  }
}

template <typename S, int D, bool FP8>
static hipError_t run_qk(const QkProblem& g, hipStream_t stream) {
  // few tokens: a workgroup each; many: a wave each, so that a vector's two loads per
  // lane and a token's angles come from the same wave's work (40 + 2 x 8 heads of 128, bf16:
  // 1024 tokens 9.8 against 12.6 us, 2048 15.6 against 14.6, 8192 55.5 against 44.9 = 5.2 TB/s)
  if (g.rows >= 2048)
    hipLaunchKernelGGL((qk_kernel<S, D, FP8, 4>), dim3(static_cast<uint32_t>((g.rows + 3) / 4)),
                       dim3(kQkThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((qk_kernel<S, D, FP8, 1>), dim3(static_cast<uint32_t>(g.rows)),
                       dim3(kQkThreads), 0, stream, g);
  return hipGetLastError();
}

template <int D>
static hipError_t run_qk_types(const QkProblem& g, hipStream_t stream) {
  if (g.dt == BDR_F32) return run_qk<float, D, false>(g, stream);
  return g.fp8 ? run_qk<uint16_t, D, true>(g, stream) : run_qk<uint16_t, D, false>(g, stream);
}

hipError_t launch_qk(const QkProblem& g, hipStream_t stream) {
  switch (g.dim) {
    case 64: return run_qk_types<64>(g, stream);
    case 128: return run_qk_types<128>(g, stream);
    default: return run_qk_types<256>(g, stream);
  }
}

}  // namespace bdr
