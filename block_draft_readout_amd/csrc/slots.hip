// Block tables and slots of a step's new tokens from the requests' lengths (gfx950).
//
// Request b holds c_b cached tokens in count_b pages and gets n_b new ones:
//   grow_b = max(0, min(width, ceil((c_b + n_b) / P)) - count_b)
// more pages, popped from the free stack in the order of the requests; a request
// with c_b < 0 is over and pushes its pages first.  Token positions and slots
// follow from the prefix sums of n_b.
//
// A few numbers per request and token: latency bounds it.  Up to 1024 requests
// one workgroup holds one per thread: one prefix sum over all that is counted,
// then pages and tokens find their request by bisection in LDS, and a token's
// page is taken from the stack rather than from the table entry that another
// thread is writing.  More requests go through in chunks of 1024.  More tokens
// than kFillRows are filled by a second launch with the whole chip.

#include <algorithm>

#include "bdr_device.h"
#include "bdr_internal.h"

namespace bdr {

struct SlotArgs {
  SlotProblem p;
  int fill;   // the planning workgroup fills the tokens' slots too
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

// Inclusive sums over the workgroup's threads of NV values, and their totals.  `red`
// has kPlanWaves slots per value; called by all threads.
template <int NV>
__device__ __forceinline__ void block_scan(int64_t (&v)[NV], int64_t (&total)[NV], int64_t* red) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = static_cast<int>(threadIdx.x) >> 6;
  const int waves = static_cast<int>(blockDim.x) >> 6;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t u = __shfl_up(v[i], d);
      if (lane >= d) v[i] += u;
    }
  }
  __syncthreads();   // an earlier use of `red` has been read
  if (lane == 63) {
#pragma unroll
    for (int i = 0; i < NV; ++i) red[i * kPlanWaves + wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    int64_t before = 0, all = 0;
    for (int w = 0; w < waves; ++w) {
      const int64_t s = red[i * kPlanWaves + w];
      if (w < wave) before += s;
      all += s;
    }
    v[i] += before;
    total[i] = all;
  }
}

__device__ __forceinline__ int32_t clamp_i32(int64_t v) {
  return static_cast<int32_t>(v < 0 ? 0 : v > 0x7FFFFFFF ? 0x7FFFFFFF : v);
}

// slot of position `pos` of a request with `count` pages, -1 where it has no page
__device__ __forceinline__ int32_t slot_of(const int32_t* row, int32_t count, int64_t pos, int32_t page) {
  const int64_t col = static_cast<uint32_t>(pos) / static_cast<uint32_t>(page);   // (positions: below 2^32)
  if (col >= count) return -1;
  const int64_t s = static_cast<int64_t>(row[col]) * page + (pos - col * page);
  return s < 0 || s > 0x7FFFFFFE ? -1 : static_cast<int32_t>(s);
}

// Token i's request: the last b with offsets[b] <= i (offsets[0] = 0, offsets[batch] > i).
__device__ __forceinline__ int32_t request_of(const int32_t* offsets, int32_t batch, int32_t i) {
  int32_t lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (offsets[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void fill_row(const SlotProblem& p, int32_t i, int32_t total) {
  int32_t pos = 0, slot = -1;
  if (i < total) {
    const int32_t b = request_of(p.offsets, p.batch, i);
    const int64_t at = static_cast<int64_t>(max(p.cached[b], 0)) + (i - p.offsets[b]);
    pos = clamp_i32(at);
    slot = slot_of(p.table + static_cast<int64_t>(b) * p.width, p.count_out[b], at, p.page);
  }
  p.positions[i] = pos;
  p.slots[i] = slot;
}

__global__ __launch_bounds__(kPlanThreads) void slot_plan_kernel(const SlotArgs g) {
  const SlotProblem& p = g.p;
  __shared__ int64_t red[4 * kPlanWaves];
  __shared__ int32_t held_s[kPlanThreads], from_s[kPlanThreads];
  __shared__ int64_t at_s[kPlanThreads];
  const int tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int64_t top0 = min(max(*p.free_count, 0), p.capacity);

  // pages that come back
  int64_t back[1] = {0}, backs[1];
  for (int b = tid; b < p.batch; b += kPlanThreads)
    if (p.cached[b] < 0) back[0] += min(max(p.count[b], 0), p.width);
  block_scan(back, backs, red);
  const int64_t R = backs[0];
  if (R > 0) {   // (uniform) the last page of the last request goes on the stack first
    int64_t base = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
      const int b = b0 + tid;
      const int held = b < p.batch && p.cached[b] < 0 ? min(max(p.count[b], 0), p.width) : 0;
      int64_t v[1] = {held}, t[1];
      block_scan(v, t, red);
      held_s[tid] = held;
      at_s[tid] = top0 + R - (base + v[0]);   // where its last page goes
      base += t[0];
      __syncthreads();
      for (int r = wave; r < min(kPlanThreads, p.batch - b0); r += kPlanWaves) {
        const int n = held_s[r];
        const int64_t to = at_s[r];
        const int32_t* row = p.table + static_cast<int64_t>(b0 + r) * p.width;
        for (int c = lane; c < n; c += 64)
          if (to + (n - 1 - c) < p.capacity) p.free_pages[to + (n - 1 - c)] = row[c];
      }
      __syncthreads();
    }
  }
  // (the stack past its capacity was not written: those pages are lost to it)
  const int64_t top = min(top0 + R, static_cast<int64_t>(p.capacity));

  int64_t tokens = 0, grown = 0, fine = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const bool live = b < p.batch;
    const int32_t c = live ? p.cached[b] : -1;
    const bool over = c < 0;
    const int32_t have = over ? 0 : min(max(p.count[b], 0), p.width);
    const int32_t n = over ? 0 : max(p.fresh[b], 0);
    const int64_t len = over ? 0 : static_cast<int64_t>(c) + n;
    const int64_t need = min((len + p.page - 1) / p.page, static_cast<int64_t>(p.width));
    const int64_t grow = max(need - have, static_cast<int64_t>(0));
    int64_t v[2] = {n, grow}, t[2];
    block_scan(v, t, red);
    const int64_t off = tokens + v[0] - n;
    const int64_t first = grown + v[1] - grow;
    const int32_t got = static_cast<int32_t>(min(max(top - first, static_cast<int64_t>(0)), grow));
    if (live) {
      p.offsets[b] = clamp_i32(off);
      p.kv_len[b] = clamp_i32(len);
      p.count_out[b] = have + got;
      const int64_t covered = min(max(static_cast<int64_t>(have + got) * p.page - c, static_cast<int64_t>(0)),
                                  static_cast<int64_t>(n));
      if (!over) fine += min(max(p.rows - off, static_cast<int64_t>(0)), covered);
    }
    tokens += t[0];
    grown += t[1];
    if (t[1] > 0) {   // (uniform)
      held_s[tid] = got;
      from_s[tid] = have;
      at_s[tid] = top - 1 - first;
      __syncthreads();
      for (int r = wave; r < min(kPlanThreads, p.batch - b0); r += kPlanWaves) {
        const int n_got = held_s[r];
        int32_t* row = p.table + static_cast<int64_t>(b0 + r) * p.width + from_s[r];
        const int64_t from = at_s[r];
        for (int i = lane; i < n_got; i += 64) row[i] = p.free_pages[from - i];
      }
      __syncthreads();
    }
  }
  int64_t f[1] = {fine}, fines[1];
  block_scan(f, fines, red);
  if (tid == 0) {
    p.offsets[p.batch] = clamp_i32(tokens);
    *p.free_out = static_cast<int32_t>(max(top - grown, static_cast<int64_t>(0)));
    *p.status = clamp_i32(tokens - fines[0]);
  }
  if (g.fill) {
    __syncthreads();   // the table, the offsets and the counts are written
    for (int i = tid; i < p.rows; i += kPlanThreads) fill_row(p, i, clamp_i32(tokens));
  }
}

// the last i in [0, n) with at[i] <= x (kPlanThreads entries, the first n ascending, at[0] <= x);
// always as many steps, so that several of them run together
template <typename I>
__device__ __forceinline__ int bisect(const I* at, int n, I x) {
  int lo = 0;
#pragma unroll
  for (int step = kPlanThreads / 2; step > 0; step >>= 1) {
    const int mid = lo + step;
    const I v = at[mid];
    lo = mid < n && v <= x ? mid : lo;
  }
  return lo;
}

constexpr int kTogether = 4;   // pages or tokens of a thread whose loads are in flight together

// At most a request per thread.
__global__ __launch_bounds__(kPlanThreads) void slot_plan_small_kernel(const SlotArgs g) {
  const SlotProblem& p = g.p;
  __shared__ int64_t red[3 * kPlanWaves];
  __shared__ int32_t off_s[kPlanThreads], start_s[kPlanThreads], have_s[kPlanThreads], count_s[kPlanThreads];
  __shared__ int64_t first_s[kPlanThreads], back_s[kPlanThreads];
  __shared__ unsigned long long fine_s;
  const int tid = static_cast<int>(threadIdx.x);
  const int threads = static_cast<int>(blockDim.x);
  const bool live = tid < p.batch;
  const int32_t c = live ? p.cached[tid] : 0;
  const int32_t held = live ? min(max(p.count[tid], 0), p.width) : 0;
  const int32_t fresh = live ? max(p.fresh[tid], 0) : 0;
  const int64_t top0 = min(max(*p.free_count, 0), p.capacity);
  const bool over = c < 0;
  const int32_t have = over ? 0 : held;
  const int32_t n = over ? 0 : fresh;
  const int64_t len = over ? 0 : static_cast<int64_t>(c) + n;
  // (len: below 2^32)
  const int64_t need = len ? min(static_cast<int64_t>((static_cast<uint32_t>(len) - 1u) / static_cast<uint32_t>(p.page)) + 1,
                                 static_cast<int64_t>(p.width))
                           : 0;
  const int64_t grow = max(need - have, static_cast<int64_t>(0));
  if (tid == 0) fine_s = 0;
  int64_t v[3] = {n, grow, over ? held : 0}, t[3];
  block_scan(v, t, red);
  const int64_t off = v[0] - n, first = v[1] - grow;
  const int64_t top = min(top0 + t[2], static_cast<int64_t>(p.capacity));
  const int32_t got = static_cast<int32_t>(min(max(top - first, static_cast<int64_t>(0)), grow));
  int64_t fine = 0;
  if (live) {
    off_s[tid] = clamp_i32(off);
    start_s[tid] = c;
    have_s[tid] = have;
    count_s[tid] = have + got;
    first_s[tid] = first;
    back_s[tid] = v[2] - (over ? held : 0);
    p.offsets[tid] = clamp_i32(off);
    p.kv_len[tid] = clamp_i32(len);
    p.count_out[tid] = have + got;
    const int64_t covered =
        min(max(static_cast<int64_t>(have + got) * p.page - max(c, 0), static_cast<int64_t>(0)), static_cast<int64_t>(n));
    fine = min(max(p.rows - off, static_cast<int64_t>(0)), covered);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) fine += __shfl_xor(fine, d);
  if ((tid & 63) == 0) atomicAdd(&fine_s, static_cast<unsigned long long>(fine));   // (whole numbers: any order)
  __syncthreads();
  if (tid == 0) {
    p.offsets[p.batch] = clamp_i32(t[0]);
    *p.free_out = static_cast<int32_t>(max(top - t[1], static_cast<int64_t>(0)));
    *p.status = clamp_i32(t[0] - static_cast<int64_t>(fine_s));
  }
  if (t[2] > 0) {   // (uniform) page i of those that come back, in the order of the table: the last goes first
    for (int64_t i0 = tid; i0 < t[2]; i0 += kTogether * threads) {
      int32_t page[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        const int64_t i = min(i0 + j * threads, t[2] - 1);
        const int b = bisect(back_s, p.batch, i);
        page[j] = p.table[static_cast<int64_t>(b) * p.width + (i - back_s[b])];
      }
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        const int64_t i = i0 + j * threads;
        const int64_t to = top0 + t[2] - 1 - i;
        if (i < t[2] && to < p.capacity) p.free_pages[to] = page[j];
      }
    }
    __syncthreads();   // the stack is whole
  }
  const int64_t given = min(t[1], top);
  for (int64_t i = tid; i < given; i += threads) {
    const int32_t page = p.free_pages[top - 1 - i];
    const int b = bisect(first_s, p.batch, i);
    p.table[static_cast<int64_t>(b) * p.width + have_s[b] + (i - first_s[b])] = page;
  }
  if (!g.fill) return;
  const int32_t total = clamp_i32(t[0]);
  for (int i0 = tid; i0 < p.rows; i0 += kTogether * threads) {
    int32_t pos[kTogether], page[kTogether], in[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int i = i0 + j * threads;
      pos[j] = 0;
      page[j] = -1;
      in[j] = 0;
      if (i < total && i < p.rows) {
        const int b = bisect(off_s, p.batch, i);
        const int64_t at = static_cast<int64_t>(start_s[b]) + (i - off_s[b]);
        const int64_t col = static_cast<uint32_t>(at) / static_cast<uint32_t>(p.page);   // (at: below 2^32)
        pos[j] = clamp_i32(at);
        in[j] = static_cast<int32_t>(at - col * p.page);
        if (col < count_s[b])
          page[j] = col < have_s[b] ? p.table[static_cast<int64_t>(b) * p.width + col]
                                    : p.free_pages[top - 1 - first_s[b] - (col - have_s[b])];
      }
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int i = i0 + j * threads;
      if (i >= p.rows) break;
      const int64_t slot = static_cast<int64_t>(page[j]) * p.page + in[j];
      p.positions[i] = pos[j];
      p.slots[i] = page[j] >= 0 && slot < 0x7FFFFFFF ? static_cast<int32_t>(slot) : -1;
    }
  }
}

__global__ __launch_bounds__(256) void slot_fill_kernel(const SlotArgs g) {
  const int32_t i = static_cast<int32_t>(blockIdx.x * 256 + threadIdx.x);
  if (i < g.p.rows) fill_row(g.p, i, g.p.offsets[g.p.batch]);
}

// Past this the rows are filled by the whole chip in a second launch (1000 requests with 1 to 64
// tokens each: 19 us, all in one workgroup 29).
constexpr int kFillRows = 4096;

hipError_t launch_slots(const SlotProblem& p, hipStream_t stream) {
  const SlotArgs g{p, p.rows <= kFillRows};
  if (p.batch <= kPlanThreads) {
    // (few waves pass their barriers sooner)
    const int threads = p.batch <= 256 && p.rows <= 1024 ? 256 : kPlanThreads;
    hipLaunchKernelGGL(slot_plan_small_kernel, dim3(1), dim3(threads), 0, stream, g);
  } else {
    hipLaunchKernelGGL(slot_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, g);
  }
  if (!g.fill) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(slot_fill_kernel, dim3((p.rows + 255) / 256), dim3(256), 0, stream, g);
  }
  return hipGetLastError();
}

}  // namespace bdr
