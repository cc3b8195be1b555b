// Row normalisation in front of the LM head, forward and backward (gfx950).
//
// Forward of row x (H features):  y = (x - mean) rstd w + b, with
//   mean = sum x / H,  rstd = (sum (x - mean)^2 / H + eps)^-1/2;
// the root-mean-square form takes mean = 0 and has no b.
// Backward, with xh = (x - mean) rstd and gy = dy w:
//   dx = rstd (gy - sum(gy) / H - xh sum(gy xh) / H)    (the sum(gy) term only
//                                                        with a mean)
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// A few flops per byte: HBM bounds both passes, so each reads its rows once.
// A row is held in registers by a group of LANES lanes (one 16-byte chunk of
// every LANES per load), so the variance is the sum of squared differences
// from the finished mean: no cancellation, no second read.  Sums are fp32;
// only the stored y, dx, dw, db are rounded to the tensors' type.
//
// The vector gradients need a sum over all rows: each workgroup of the
// backward pass walks its share of the rows with the column sums in
// registers, joins its groups' sums in LDS in group order and writes one fp32
// partial row; a second launch adds the partial rows in order.  No atomics:
// the same inputs give the same bits.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "bdr_internal.h"
#include "train_device.h"

namespace bdr {

struct NormArgs {
  const void* x;
  int64_t rows, x_stride, dy_stride;
  int hidden;
  const void* dy;
  const void* w;
  const void* b;
  float eps, inv_h;
  void* y;              // forward output, backward dx
  float* mean;          // forward: written where not NULL; backward: read
  float* rstd;
  float* partial;       // backward: [groups][2][H] (dw, db) column sums
  int want_dx, want_dw, want_db;
};

template <typename S>
__device__ __forceinline__ void unpack16(u32x4_t v, float (&f)[Elem<S>::PER16]) {
  if constexpr (sizeof(S) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(v[e] << 16);
      f[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(v[e]);
  }
}

template <typename S>
__device__ __forceinline__ u32x4_t pack16(const float (&f)[Elem<S>::PER16]) {
  u32x4_t v;
  if constexpr (sizeof(S) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(f[e]);
  }
  return v;
}

// Sums of the group of LANES lanes a thread belongs to, in every lane.  `red`
// has one slot per wave for each value; called by all threads of the workgroup.
template <int LANES, int NV>
__device__ __forceinline__ void group_sums(float (&v)[NV], float* red, int waves) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if constexpr (LANES > 64) {
    const int wave = static_cast<int>(threadIdx.x) >> 6;
    __syncthreads();   // an earlier use of `red` has been read
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) red[i * waves + wave] = v[i];
    }
    __syncthreads();
    const int w0 = static_cast<int>(threadIdx.x) / LANES * (LANES / 64);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < LANES / 64; ++w) s += red[i * waves + w0 + w];
      v[i] = s;
    }
  }
}

constexpr int kFwdThreads = 256;

template <typename S, int LANES, int CH>
__global__ __launch_bounds__(kFwdThreads) void norm_forward_kernel(const NormArgs g) {
  constexpr int PER = Elem<S>::PER16;
  __shared__ float red[kFwdThreads / 64];
  const int lane = static_cast<int>(threadIdx.x) % LANES;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kFwdThreads / LANES) +
                      static_cast<int>(threadIdx.x) / LANES;
  const bool live = row < g.rows;
  const S* x = static_cast<const S*>(g.x) + (live ? row : 0) * g.x_stride;
  const S* wv = static_cast<const S*>(g.w);
  const S* bv = static_cast<const S*>(g.b);
  u32x4_t raw[CH], rw[CH], rb[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * LANES + lane) * PER;
    const bool in = col < g.hidden;
    raw[c] = in ? load16(x + col) : u32x4_t{0, 0, 0, 0};
    rw[c] = in ? load16(wv + col) : u32x4_t{0, 0, 0, 0};
    rb[c] = in && bv ? load16(bv + col) : u32x4_t{0, 0, 0, 0};
  }
  float mean = 0.f;
  if (g.mean) {
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float f[PER];
      unpack16<S>(raw[c], f);
#pragma unroll
      for (int e = 0; e < PER; ++e) s[0] += f[e];   // columns past H hold zeros
    }
    group_sums<LANES>(s, red, kFwdThreads / 64);
    mean = s[0] * g.inv_h;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if ((c * LANES + lane) * PER < g.hidden) {
      float f[PER];
      unpack16<S>(raw[c], f);
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const float d = f[e] - mean;
        q[0] += d * d;
      }
    }
  }
  group_sums<LANES>(q, red, kFwdThreads / 64);
  const float rstd = 1.0f / sqrtf(q[0] * g.inv_h + g.eps);
  if (!live) return;
  if (lane == 0) {
    if (g.mean) g.mean[row] = mean;
    g.rstd[row] = rstd;
  }
  S* y = static_cast<S*>(g.y) + row * g.hidden;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * LANES + lane) * PER;
    if (col < g.hidden) {
      float f[PER], w[PER], b[PER];
      unpack16<S>(raw[c], f);
      unpack16<S>(rw[c], w);
      unpack16<S>(rb[c], b);
#pragma unroll
      for (int e = 0; e < PER; ++e) f[e] = (f[e] - mean) * rstd * w[e] + b[e];
      *reinterpret_cast<u32x4_t*>(y + col) = pack16<S>(f);
    }
  }
}

constexpr int kBwdThreads = 512;

template <typename S, int LANES, int CH>
__global__ __launch_bounds__(kBwdThreads) void norm_backward_kernel(const NormArgs g) {
  constexpr int PER = Elem<S>::PER16;
  constexpr int GROUPS = kBwdThreads / LANES;
  constexpr int WAVES = kBwdThreads / 64;
  __shared__ float red[2 * WAVES];
  extern __shared__ float cols[];   // [H], the groups' column sums joined
  const int lane = static_cast<int>(threadIdx.x) % LANES;
  const int group = static_cast<int>(threadIdx.x) / LANES;
  const S* wv = static_cast<const S*>(g.w);
  u32x4_t rw[CH];
  float dw[CH][PER], db[CH][PER];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * LANES + lane) * PER;
    rw[c] = col < g.hidden ? load16(wv + col) : u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < PER; ++e) dw[c][e] = db[c][e] = 0.f;
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x) * GROUPS;
  // A group of several waves holds the next row's chunks while it works on one
  // (its joins are barriers, and few rows are in flight); waves by themselves
  // cover each other.
  constexpr bool kAhead = LANES > 64;
  u32x4_t rx[CH], rd[CH], nx[kAhead ? CH : 1], nd[kAhead ? CH : 1];
  auto load_row = [&](int64_t row, u32x4_t* vx, u32x4_t* vd) {
    const bool live = row < g.rows;
    const S* x = static_cast<const S*>(g.x) + (live ? row : 0) * g.x_stride;
    const S* dy = static_cast<const S*>(g.dy) + (live ? row : 0) * g.dy_stride;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * LANES + lane) * PER;
      const bool in = live && col < g.hidden;
      vx[c] = in ? load16(x + col) : u32x4_t{0, 0, 0, 0};
      vd[c] = in ? load16(dy + col) : u32x4_t{0, 0, 0, 0};
    }
  };
  if constexpr (kAhead) load_row(static_cast<int64_t>(blockIdx.x) * GROUPS + group, nx, nd);
  // every group walks the same number of rounds: the joins below hold barriers
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * GROUPS; r0 < g.rows; r0 += stride) {
    const int64_t row = r0 + group;
    const bool live = row < g.rows;
    if constexpr (kAhead) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        rx[c] = nx[c];
        rd[c] = nd[c];
      }
      load_row(row + stride, nx, nd);
    } else {
      load_row(row, rx, rd);
    }
    const float mean = g.mean && live ? g.mean[row] : 0.f;
    const float rstd = live ? g.rstd[row] : 0.f;
    float s[2] = {0.f, 0.f};   // sum gy, sum gy xh
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float f[PER], d[PER], w[PER];
      unpack16<S>(rx[c], f);
      unpack16<S>(rd[c], d);
      unpack16<S>(rw[c], w);
#pragma unroll
      for (int e = 0; e < PER; ++e) {   // dy is zero past H and past the last row
        const float xh = (f[e] - mean) * rstd;
        const float gy = d[e] * w[e];
        s[0] += gy;
        s[1] += gy * xh;
        dw[c][e] += d[e] * xh;
        db[c][e] += d[e];
      }
    }
    if (g.want_dx) {
      group_sums<LANES>(s, red, WAVES);
      const float m1 = g.mean ? s[0] * g.inv_h : 0.f;
      const float m2 = s[1] * g.inv_h;
      if (live) {
        S* dx = static_cast<S*>(g.y) + row * g.hidden;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int col = (c * LANES + lane) * PER;
          if (col < g.hidden) {
            float f[PER], d[PER], w[PER];
            unpack16<S>(rx[c], f);
            unpack16<S>(rd[c], d);
            unpack16<S>(rw[c], w);
#pragma unroll
            for (int e = 0; e < PER; ++e) {
              const float xh = (f[e] - mean) * rstd;
              f[e] = rstd * (d[e] * w[e] - m1 - xh * m2);
            }
            *reinterpret_cast<u32x4_t*>(dx + col) = pack16<S>(f);
          }
        }
      }
    }
  }
  // join the groups' column sums in group order: dw, then db
  static_for<2>([&](auto which) {
    constexpr int k = decltype(which)::value;
    if (k == 0 ? g.want_dw : g.want_db) {
      for (int gr = 0; gr < GROUPS; ++gr) {
        __syncthreads();
        if (group == gr) {
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const int col = (c * LANES + lane) * PER;
            if (col < g.hidden) {
#pragma unroll
              for (int e = 0; e < PER; ++e) {
                const float v = k == 0 ? dw[c][e] : db[c][e];
                cols[col + e] = gr == 0 ? v : cols[col + e] + v;
              }
            }
          }
        }
      }
      __syncthreads();
      float* out = g.partial + (2 * static_cast<int64_t>(blockIdx.x) + k) * g.hidden;
      for (int i = static_cast<int>(threadIdx.x); i < g.hidden; i += kBwdThreads) out[i] = cols[i];
    }
  });
}

// dw / db: the partial rows added in order, 16 interleaved sums per column
// joined through LDS.  Grid (ceil(H / 64), 2), 1024 threads.
template <typename S>
__global__ __launch_bounds__(1024) void norm_vector_grad_kernel(const float* partial, int n_part,
                                                                int hidden, S* dw, S* db) {
  __shared__ float sums[16][64];
  const int k = static_cast<int>(blockIdx.y);
  S* out = k == 0 ? dw : db;
  if (!out) return;   // whole workgroup
  const int c = static_cast<int>(threadIdx.x) & 63;
  const int p = static_cast<int>(threadIdx.x) >> 6;
  const int col = static_cast<int>(blockIdx.x) * 64 + c;
  float s = 0.f;
  if (col < hidden)
#pragma unroll 4
    for (int i = p; i < n_part; i += 16) s += partial[(2 * static_cast<int64_t>(i) + k) * hidden + col];
  sums[p][c] = s;
  __syncthreads();
  if (p == 0 && col < hidden) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sums[i][c];
    out[col] = rounded<S>(t);
  }
}

// Workgroups of the backward pass: one per compute unit; each writes a partial row.
static int64_t norm_backward_blocks(int64_t rows) {
  return std::max<int64_t>(1, std::min<int64_t>(256, (rows + 3) / 4));
}

size_t norm_workspace(int64_t rows, int64_t hidden) {
  return align256(static_cast<size_t>(norm_backward_blocks(rows)) * 2 * hidden * sizeof(float));
}

// f(integral_constant CH) for the smallest of the listed chunk counts that holds ch
template <int FIRST, int... REST, typename F>
static hipError_t by_chunks(int64_t ch, F&& f) {
  if constexpr (sizeof...(REST) == 0)
    return f(std::integral_constant<int, FIRST>{});
  else
    return ch <= FIRST ? f(std::integral_constant<int, FIRST>{}) : by_chunks<REST...>(ch, f);
}

// A wave holds a row of up to 256 chunks of 16 bytes by itself, 256 lanes a
// longer one.
template <typename S>
static hipError_t norm_forward(const NormArgs& g, hipStream_t stream) {
  const int64_t chunks = g.hidden / Elem<S>::PER16;
  auto run = [&](auto lanes, auto ch) {
    constexpr int LANES = decltype(lanes)::value;
    constexpr int CH = decltype(ch)::value;
    constexpr int RPB = kFwdThreads / LANES;
    hipLaunchKernelGGL((norm_forward_kernel<S, LANES, CH>),
                       dim3(static_cast<unsigned>((g.rows + RPB - 1) / RPB)), dim3(kFwdThreads), 0,
                       stream, g);
    return hipGetLastError();
  };
  std::integral_constant<int, 64> wave;
  std::integral_constant<int, 256> wide;
  if (chunks <= 4 * 64)
    return by_chunks<1, 2, 3, 4>((chunks + 63) / 64, [&](auto ch) { return run(wave, ch); });
  if constexpr (sizeof(S) == 4)   // rows over 8192
    if (chunks > 8 * 256) return run(wide, std::integral_constant<int, 16>{});
  return by_chunks<2, 3, 4, 8>((chunks + 255) / 256, [&](auto ch) { return run(wide, ch); });
}

// A wave walks rows of up to 2560 features (fp32: 2048) by itself: no barriers,
// and a workgroup's eight waves have as many rows in flight (16381 x 2560 bf16:
// 50 us, 256 lanes a row 68 us).  Longer rows, whose column sums would not
// fit a wave's registers, are spread over 256 or 512 lanes.
template <typename S>
static hipError_t norm_backward(const NormArgs& g, void* dw, void* db, hipStream_t stream) {
  const int64_t chunks = g.hidden / Elem<S>::PER16;
  const unsigned blocks = static_cast<unsigned>(norm_backward_blocks(g.rows));
  const size_t lds = g.want_dw || g.want_db ? static_cast<size_t>(g.hidden) * 4 : 0;
  auto run = [&](auto lanes, auto ch) {
    hipLaunchKernelGGL((norm_backward_kernel<S, decltype(lanes)::value, decltype(ch)::value>),
                       dim3(blocks), dim3(kBwdThreads), lds, stream, g);
    return hipGetLastError();
  };
  std::integral_constant<int, 64> wave;
  std::integral_constant<int, 256> wide;
  std::integral_constant<int, 512> whole;
  const int64_t ch = (chunks + 63) / 64;
  auto wide_run = [&](auto c) { return run(wide, c); };
  hipError_t e;
  if constexpr (sizeof(S) == 2) {
    if (ch <= 5)
      e = by_chunks<1, 2, 3, 4, 5>(ch, [&](auto c) { return run(wave, c); });
    else if (chunks <= 4 * 256)
      e = by_chunks<2, 3, 4>((chunks + 255) / 256, wide_run);
    else
      e = run(whole, std::integral_constant<int, 4>{});
  } else {
    if (ch <= 8)
      e = by_chunks<1, 2, 3, 4, 6, 8>(ch, [&](auto c) { return run(wave, c); });
    else if (chunks <= 6 * 256)
      e = by_chunks<3, 4, 5, 6>((chunks + 255) / 256, wide_run);
    else
      e = by_chunks<4, 8>((chunks + 511) / 512, [&](auto c) { return run(whole, c); });
  }
  if (e != hipSuccess || !(dw || db)) return e;
  hipLaunchKernelGGL(norm_vector_grad_kernel<S>, dim3(static_cast<unsigned>((g.hidden + 63) / 64), 2),
                     dim3(1024), 0, stream, g.partial, static_cast<int>(blocks), g.hidden,
                     static_cast<S*>(dw), static_cast<S*>(db));
  return hipGetLastError();
}

hipError_t launch_norm(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, bdr_dtype dt,
                       const void* w, const void* b, float eps, void* y, float* mean, float* rstd,
                       hipStream_t stream) {
  NormArgs g{};
  g.x = x;
  g.rows = rows;
  g.x_stride = x_stride;
  g.hidden = static_cast<int>(hidden);
  g.w = w;
  g.b = b;
  g.eps = eps;
  g.inv_h = 1.0f / static_cast<float>(hidden);
  g.y = y;
  g.mean = mean;
  g.rstd = rstd;
  return dt == BDR_BF16 ? norm_forward<uint16_t>(g, stream) : norm_forward<float>(g, stream);
}

hipError_t launch_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                int64_t rows, int64_t hidden, bdr_dtype dt, const void* w,
                                const float* mean, const float* rstd, void* dx, void* dw, void* db,
                                void* workspace, hipStream_t stream) {
  NormArgs g{};
  g.x = x;
  g.rows = rows;
  g.x_stride = x_stride;
  g.dy_stride = dy_stride;
  g.hidden = static_cast<int>(hidden);
  g.dy = dy;
  g.w = w;
  g.inv_h = 1.0f / static_cast<float>(hidden);
  g.y = dx;
  g.mean = const_cast<float*>(mean);
  g.rstd = const_cast<float*>(rstd);
  g.partial = static_cast<float*>(workspace);
  g.want_dx = dx != nullptr;
  g.want_dw = dw != nullptr;
  g.want_db = db != nullptr;
  return dt == BDR_BF16 ? norm_backward<uint16_t>(g, dw, db, stream)
                        : norm_backward<float>(g, dw, db, stream);
}

}  // namespace bdr
