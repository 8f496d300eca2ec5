// Block tables, positions and cache slots of a step's new tokens (bl_page_map),
// from the requests' lengths and counts:
//   total = length + count;  ask = max(0, ceil(total / page) - owned);
//   the k-th page asked for, in the order of the requests, is free[free_count - 1 - k];
//   token i of request r: position = length + i - start[r],
//   slot = table[r][position / page] * page + position % page.
// The pages of requests that end go back on top of the stack.
//
// Everything hangs on prefix sums over the requests, so one CTA scans them (1024
// at a time) and writes the tables; when there are many tokens, the other CTAs of
// its cluster share the slots.  Pages are pushed only after all have been popped.
//
// Bound: latency (a few dependent reads of some KB, the barriers of the scan, a binary search per token in shared
// memory): 64 requests with a token each 4.4 us; 256 requests, 12 of them prompts, 8200 tokens 7.8 us.  Scans of a
// warp's sums by one thread and searches in global memory took 5.7 and 9.7 us.
#include "bl_device.cuh"
#include "bl_internal.h"
#include "paged.cuh"

namespace bl {
namespace {

constexpr int kThreads = 1024;
constexpr int kCached = 2048;  // requests whose starts and old lengths are kept in shared memory

struct Args {
  const int32_t *length, *count, *owned, *free_count;
  int32_t *table, *free_pages, *start, *position, *slot, *length_out, *owned_out, *free_left;
  int64_t R, W, pages, M;
  int page;
  unsigned int* err;
};

struct Three {
  int64_t ask, tokens, give;
};
__device__ __forceinline__ Three operator+(Three a, Three b) { return {a.ask + b.ask, a.tokens + b.tokens, a.give + b.give}; }

__device__ __forceinline__ Three shift_up(Three v, int o) {
  return {__shfl_up_sync(0xffffffffu, v.ask, o), __shfl_up_sync(0xffffffffu, v.tokens, o), __shfl_up_sync(0xffffffffu, v.give, o)};
}
__device__ __forceinline__ Three of_lane(Three v, int l) {
  return {__shfl_sync(0xffffffffu, v.ask, l), __shfl_sync(0xffffffffu, v.tokens, l), __shfl_sync(0xffffffffu, v.give, l)};
}
__device__ __forceinline__ Three scan_lanes(Three v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Three w = shift_up(v, o);
    if (int(threadIdx.x & 31) >= o) v = v + w;
  }
  return v;
}

// Sum over the threads before this one; `total` receives that of all.
__device__ __forceinline__ Three scan_before(Three v, Three* warps, Three& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Three through = scan_lanes(v);
  __syncthreads();  // the last scan's sums have been read
  if (lane == 31) warps[warp] = through;
  __syncthreads();
  const Three up_to = scan_lanes(warps[lane]);
  total = of_lane(up_to, 31);
  const Three before = of_lane(up_to, max(warp - 1, 0));
  const int64_t has = warp > 0;
  return {has * before.ask + through.ask - v.ask, has * before.tokens + through.tokens - v.tokens, has * before.give + through.give - v.give};
}

// A request's own numbers, its arguments brought into range.
struct Request {
  int64_t total, ask;
  int owned, count;
  bool ends, bad;
};
__device__ __forceinline__ Request request_of(const Args& a, int64_t r) {
  Request q = {0, 0, 0, 0, false, false};
  if (r >= a.R) return q;
  const int length = a.length[r], count = a.count[r], owned = a.owned[r];
  q.ends = count < 0;
  q.count = max(count, 0);
  q.owned = int(max(int64_t(0), min(int64_t(owned), a.W)));
  q.bad = length < 0 || q.owned != owned;
  q.total = q.ends ? 0 : int64_t(max(length, 0)) + q.count;
  int64_t need = (q.total + a.page - 1) / a.page;
  if (need > a.W || q.total >= INT32_MAX) q.bad = true;
  need = min(need, a.W);
  q.ask = q.ends ? 0 : max(int64_t(0), need - q.owned);
  return q;
}

// A request's tokens before the step, from its new length; -1: its positions do not fit, so that its tokens have none.
__device__ __forceinline__ int old_length(int length, int count) { return length == INT32_MAX ? -1 : length - max(count, 0); }

// f(x, y, j) for j = 0..n-1 of every lane's (n, x, y), lane by lane, by the whole converged warp.
template <class F>
__device__ __forceinline__ void each_page(int64_t n, int64_t x, int64_t y, F f) {
  const int lane = threadIdx.x & 31;
  unsigned todo = __ballot_sync(0xffffffffu, n > 0);
  while (todo) {
    const int from = __ffs(todo) - 1;
    todo &= todo - 1;
    const int64_t many = __shfl_sync(0xffffffffu, n, from);
    const int64_t xf = __shfl_sync(0xffffffffu, x, from), yf = __shfl_sync(0xffffffffu, y, from);
    for (int64_t j = lane; j < many; j += 32) f(xf, yf, j);
    __syncwarp();
  }
}

template <int C>
__global__ void __launch_bounds__(kThreads) page_map_kernel(const Args a) {
  __shared__ Three warps[kThreads / 32];
  __shared__ int starts[kCached + 1], old[kCached];
  const int tid = threadIdx.x;
  const uint32_t rank = C == 1 ? 0 : cluster_ctarank();
  bool bad = false;
  pdl_wait();
  if (rank == 0) {
    const int given = a.free_count[0];
    const int64_t free_count = max(int64_t(0), min(int64_t(given), a.pages));
    bad = given != free_count;
    Three sum = {0, 0, 0}, part;
    bool ends = false;
    for (int64_t base = 0; base < a.R; base += kThreads) {
      const int64_t r = base + tid;
      const Request q = request_of(a, r);
      const Three mine = sum + scan_before({q.ask, q.count, q.ends ? q.owned : 0}, warps, part);
      sum = sum + part;
      const int64_t got = max(int64_t(0), min(q.ask, free_count - mine.ask));
      bad |= q.bad || got < q.ask;
      ends |= q.ends;
      if (r < a.R) {
        a.start[r] = int(min(mine.tokens, a.M));
        if (r < kCached) {
          starts[r] = int(min(mine.tokens, a.M));
          old[r] = old_length(int(min(q.total, int64_t(INT32_MAX))), q.count);
        }
        a.length_out[r] = int(min(q.total, int64_t(INT32_MAX)));
        if (!q.ends) a.owned_out[r] = q.owned + int(got);
      }
      // most requests ask for one page at most
      const int64_t row = r * a.W + q.owned;
      if (q.ask > 0) a.table[row] = mine.ask < free_count ? a.free_pages[free_count - 1 - mine.ask] : -1;
      each_page(q.ask - 1, mine.ask + 1, row + 1, [&](int64_t k, int64_t to, int64_t j) {
        a.table[to + j] = k + j < free_count ? a.free_pages[free_count - 1 - k - j] : -1;
      });
    }
    bad |= sum.tokens > a.M;
    const int64_t left = free_count - min(sum.ask, free_count);
    if (__syncthreads_or(ends)) {  // every page has been popped
      Three before = {0, 0, 0};
      for (int64_t base = 0; base < a.R; base += kThreads) {
        const int64_t r = base + tid;
        // owned_out may be owned: of a request that ends it has not been written yet
        const bool over = r < a.R && a.count[r] < 0;
        const int owned = over ? int(max(int64_t(0), min(int64_t(a.owned[r]), a.W))) : 0;
        const Three mine = before + scan_before({0, 0, owned}, warps, part);
        before = before + part;
        if (over) a.owned_out[r] = 0;
        const int64_t to = left + mine.give, row = r * a.W;
        each_page(owned, to, row, [&](int64_t at, int64_t entry, int64_t j) {
          if (at + j < a.pages) a.free_pages[at + j] = a.table[entry + j];
        });
      }
    }
    bad |= left + sum.give > a.pages;
    if (tid == 0) {
      a.start[a.R] = int(min(sum.tokens, a.M));
      if (a.R <= kCached) starts[a.R] = int(min(sum.tokens, a.M));
      a.free_left[0] = int(min(left + sum.give, a.pages));
    }
  }
  if (C > 1) {
    __syncwarp();
    cluster_sync();
  }
  const bool cached = a.R <= kCached;
  if (cached && rank != 0) {
    for (int r = tid; r <= a.R; r += kThreads) {
      starts[r] = a.start[r];
      if (r < a.R) old[r] = old_length(a.length_out[r], a.count[r]);
    }
  }
  __syncthreads();
  const int* start = cached ? starts : a.start;
  const int last = start[a.R];
  for (int64_t i = int64_t(rank) * kThreads + tid; i < a.M; i += C * kThreads) {
    int position = -1, slot = -1;
    if (i < last) {
      const int64_t r = request_of_token(start, a.R, int(i));
      const int before = cached ? old[r] : old_length(a.length_out[r], a.count[r]);
      if (before >= 0) {
        position = before + int(i) - start[r];
        const int entry = position / a.page;
        const int page = entry < a.W ? a.table[r * a.W + entry] : -1;
        if (page >= 0 && page < a.pages) slot = page * a.page + position % a.page;
        bad |= page >= a.pages;
      }
    }
    a.position[i] = position;
    a.slot[i] = slot;
  }
  if (__syncthreads_or(bad) && tid == 0) atomicOr(a.err, BL_DEVERR_RANGE);
  pdl_launch_dependents();
}

}  // namespace

cudaError_t launch_page_map(const int32_t* length, const int32_t* count, int32_t* table, const int32_t* owned,
                            int32_t* free_pages, const int32_t* free_count, int64_t R, int64_t W, int64_t pages, int page,
                            int64_t M, int32_t* start, int32_t* position, int32_t* slot, int32_t* length_out,
                            int32_t* owned_out, int32_t* free_left, cudaStream_t s) {
  unsigned int* err = dev_error_ptr();
  if (!err) return cudaErrorUnknown;
  const Args a{length, count, owned, free_count, table, free_pages, start, position, slot, length_out, owned_out, free_left,
               R, W, pages, M, page, err};
  const bool pdl = overlap_enabled();
  if (M <= 2 * kThreads) return launch(page_map_kernel<1>, dim3(1), dim3(kThreads), 0, s, pdl, a);
  return launch_cluster(page_map_kernel<8>, 8, dim3(8), dim3(kThreads), 0, s, pdl, a);
}

}  // namespace bl
