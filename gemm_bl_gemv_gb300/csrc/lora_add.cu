// Low-rank adapters of many requests beside a shared product (bl_lora_add):
//   y[m,n] = base[m,n] + scale[a] * sum_r B[a,n,r] (sum_k A[a,r,k] x[m,k]),
// a = adapter[m], negative for none.  This file has the kernel for scattered
// tokens (a decode step: every token has its own adapter); tiles of 128 tokens
// with few runs of one adapter go to lora_tile.cu when there are many.
//
// A cluster of 8 CTAs takes up to four neighbouring tokens of one adapter.
// Each CTA forms the inner products with an eighth of K, a warp a row of A at
// a time; the eighths meet through distributed shared memory, added in rank
// order; then each CTA forms an eighth of the outputs, a thread a row of B.
// The CTA's part of B and of base is fetched into L2 while A is being read, so
// that they come from HBM in one stream.  All sums are fp32.
//
// Bound: latency: launch, adapter -> A, the cluster's exchange, B, each a
// dependent step of one to three us (one token, 2560 -> 6912, rank 16: 5.1 us;
// 64 tokens over 40 adapters, 5120 -> 13824, rank 32: 20.6 us, a third of HBM's
// rate for the 47 MB that they need).
#include <algorithm>

#include "bl_internal.h"
#include "lora.cuh"

namespace bl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kParts = 8;      // CTAs of a cluster
constexpr int64_t kOnePerCluster = 256;  // tokens up to which each has a cluster
constexpr int64_t kTileTokens = 257;  // tokens from which the tiles' kernel is launched as well
static_assert(kTileTokens > kOnePerCluster, "beside the tiles a cluster takes a group of tokens");
constexpr int kPerSm = 4;      // CTAs of an SM
constexpr int kBatch = 256;    // tiles looked at together
constexpr int kGroup = 4;      // tokens that share the reads of an adapter

struct Args {
  const void* x;
  const int32_t* adapter;
  const uint16_t *a, *b;
  const float* scale;
  const void* base;
  void* y;
  unsigned int* err;
  int64_t M, N, K, L;
  int R;
  int per;     // tokens of a cluster
};

struct __align__(16) Shared {
  float part[2][kGroup][128];  // this CTA's share of the inner products; every second run uses the other half
  float low[kGroup][128];
  uint32_t scattered[kBatch / 32];  // bit i: tile batch + i is this kernel's
};

// The groups of tokens in tiles of many runs, of which this cluster takes every `clusters`-th: the other kernel has
// the rest, and a cluster for each of them, with nothing to do, would take longer than looking (8192 tokens: 10 us).
struct Scattered {
  const Args& g;
  Shared& sh;
  int clusters, group, word;
  uint32_t bits;
  int64_t batch, tile;
  __device__ __forceinline__ Scattered(const Args& args, Shared& shared, int cluster, int n)
      : g(args), sh(shared), clusters(n), group(cluster - n), word(kBatch / 32), bits(0), batch(-kBatch), tile(-1) {}
  __device__ void look() {  // a warp a tile
    const int lane = threadIdx.x & 31;
    __syncthreads();
    if (threadIdx.x < kBatch / 32) sh.scattered[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < kBatch && (batch + i) * kTile < g.M; i += kWarps) {
      int starts = 0;
#pragma unroll
      for (int j = 0; j < kTile / 32; ++j) {
        const int64_t t = (batch + i) * kTile + 32 * j + lane;
        const bool start = t < g.M && ((j == 0 && lane == 0) || adapter_of(g.adapter, t, g.L) != adapter_of(g.adapter, t - 1, g.L));
        starts += __popc(__ballot_sync(0xffffffffu, start));
      }
      if (lane == 0 && starts > kTileRuns) atomicOr(&sh.scattered[i >> 5], 1u << (i & 31));
    }
    __syncthreads();
  }
  __device__ __forceinline__ bool next_tile() {
    while (bits == 0) {
      if (++word < kBatch / 32) {
        bits = sh.scattered[word];
        continue;
      }
      batch += kBatch;
      if (batch * kTile >= g.M) return false;
      look();
      word = -1;
    }
    tile = batch + word * 32 + __ffs(bits) - 1;
    bits &= bits - 1;
    return true;
  }
  // The first token of the next group, -1 behind the last.
  __device__ __forceinline__ int64_t next() {
    constexpr int kGroups = kTile / kGroup;
    group += clusters;
    if (tile < 0 && !next_tile()) return -1;
    for (; group >= kGroups; group -= kGroups)
      if (!next_tile()) return -1;
    return tile * kTile + group * kGroup;
  }
};

// This CTA's share of the inner products of NT tokens from m on with A[l].  A
// warp reads kRows rows of A at a time (kRows divides R).
template <bool XB, int NT, int kRows>
__device__ __forceinline__ void down(const Args& g, float (*part)[128], int64_t m, int nt, int64_t l, uint32_t me) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = int(g.K / 8), per = (chunks + kParts - 1) / kParts;
  const int c0 = min(int(me) * per, chunks), c1 = min(c0 + per, chunks);
  for (int r0 = warp * kRows; r0 < g.R; r0 += kWarps * kRows) {
    const uint4* rows = reinterpret_cast<const uint4*>(g.a) + (l * g.R + r0) * chunks;
    float acc[kRows][NT] = {};
    for (int c = c0 + lane; c < c1; c += 32) {
      uint4 q[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) q[r] = rows[int64_t(r) * chunks + c];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (NT > 1 && t >= nt) break;
        float xv[8];
        load8<XB>(g.x, (m + t) * chunks + c, xv);
#pragma unroll
        for (int r = 0; r < kRows; ++r) acc[r][t] = dot8(q[r], xv, acc[r][t]);
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (NT > 1 && t >= nt) break;
        const float v = warp_sum(acc[r][t]);
        if (lane == 0) part[t][r0 + r] = v;
      }
  }
}

// This CTA's outputs [n0, n1) of NT tokens: a thread a row of B, two rows at a time.
template <bool YB, int NT>
__device__ __forceinline__ void up(const Args& g, const float (*low)[128], int64_t m, int nt, const uint16_t* b,
                                   int64_t n0, int64_t n1) {
  const int r8 = g.R / 8;
  for (int64_t n = n0 + threadIdx.x; n < n1; n += 2 * kThreads) {
    const bool two = n + kThreads < n1;
    const uint4* row0 = reinterpret_cast<const uint4*>(b + n * g.R);
    const uint4* row1 = two ? row0 + int64_t(kThreads) * r8 : row0;
    float acc0[NT] = {}, acc1[NT] = {}, add0[NT], add1[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (NT == 1 || t < nt) {
        const int64_t i = (m + t) * g.N + n;
        add0[t] = load1<YB>(g.base, i);
        add1[t] = two ? load1<YB>(g.base, i + kThreads) : 0.f;
      }
#pragma unroll 4
    for (int r = 0; r < r8; ++r) {
      const uint4 q0 = row0[r], q1 = row1[r];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float4 f0 = *reinterpret_cast<const float4*>(&low[t][8 * r]);
        const float4 f1 = *reinterpret_cast<const float4*>(&low[t][8 * r + 4]);
        const float v[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
        acc0[t] = dot8(q0, v, acc0[t]);
        acc1[t] = dot8(q1, v, acc1[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (NT > 1 && t >= nt) break;
      const int64_t i = (m + t) * g.N + n;
      store1<YB>(g.y, i, add0[t] + acc0[t]);
      if (two) store1<YB>(g.y, i + kThreads, add1[t] + acc1[t]);
    }
  }
}

// TILES: tiles of few runs are another kernel's.
template <bool XB, bool YB, bool TILES>
__global__ void __launch_bounds__(kThreads, kPerSm) lora_token_kernel(const Args g) {
  __shared__ Shared sh;
  const uint32_t me = cluster_ctarank();
  const int cluster = int(blockIdx.x / kParts);
  if (TILES)
    __threadfence();  // the tiles' kernel has waited, fenced and started this one, which runs beside it
  else
    pdl_wait();
  Scattered units(g, sh, cluster, int(gridDim.x / kParts));
  const int64_t n_part = (g.N + kParts - 1) / kParts, n0 = int64_t(me) * n_part, n1 = min(n0 + n_part, g.N);
  int run = 0;
  int64_t m = TILES ? units.next() : int64_t(cluster) * g.per, last = min(m + g.per, g.M);
  while (m >= 0) {
    if (m >= last) {
      m = TILES ? units.next() : -1;
      last = min(m + g.per, g.M);
      continue;
    }
    // the first of the tokens with this adapter among four aligned ones, and how many follow
    const int l = adapter_of(g.adapter, m, g.L);
    const int64_t end = min(g.M, (m / kGroup + 1) * kGroup);
    if (m % kGroup != 0 && adapter_of(g.adapter, m - 1, g.L) == l) {
      ++m;
      continue;
    }
    int nt = 1;
    while (m + nt < end && adapter_of(g.adapter, m + nt, g.L) == l) ++nt;
    if (me == 0 && threadIdx.x < nt && g.adapter[m + threadIdx.x] >= g.L && g.err) atomicOr(g.err, BL_DEVERR_RANGE);
    if (l < 0) {
      if (g.y != g.base)
        for (int t = 0; t < nt; ++t)
          for (int64_t n = n0 + threadIdx.x; n < n1; n += kThreads)
            store1<YB>(g.y, (m + t) * g.N + n, load1<YB>(g.base, (m + t) * g.N + n));
      m += nt;
      continue;
    }
    const uint16_t* b = g.b + int64_t(l) * g.N * g.R;
    for (int64_t i = n0 * g.R + int64_t(threadIdx.x) * 64; i < n1 * g.R; i += kThreads * 64)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(b + i));
    for (int t = 0; t < nt; ++t) {
      constexpr int kSize = YB ? 2 : 4;
      const char* at = static_cast<const char*>(g.base) + (m + t) * g.N * kSize;
      for (int64_t i = n0 * kSize + int64_t(threadIdx.x) * 128; i < n1 * kSize; i += kThreads * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i));
    }
    float(*part)[128] = sh.part[run & 1];
    if (nt > 1)
      down<XB, kGroup, 2>(g, part, m, nt, l, me);
    else if (g.R <= 16)
      down<XB, 1, 2>(g, part, m, nt, l, me);
    else
      down<XB, 1, 4>(g, part, m, nt, l, me);
    __syncwarp();  // the cluster barrier wants converged warps
    cluster_sync();
    for (int i = threadIdx.x; i < nt * g.R; i += kThreads) {
      const int t = i / g.R, r = i % g.R;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kParts; ++q) v += *peer(&part[t][r], q);
      sh.low[t][r] = v * g.scale[l];
    }
    __syncthreads();
    if (nt > 1)
      up<YB, kGroup>(g, sh.low, m, nt, b, n0, n1);
    else
      up<YB, 1>(g, sh.low, m, nt, b, n0, n1);
    __syncthreads();  // the last use of low
    ++run;
    m += nt;
  }
  // another CTA may still read this one's share (after two runs the barrier between them has settled it)
  __syncwarp();
  if (run > 0) cluster_sync();
  if (TILES && blockIdx.x == 0) pdl_wait();  // this kernel's end is the call's end
  pdl_launch_dependents();
}

template <bool XB, bool YB, bool TILES>
cudaError_t launch_tokens(const Args& g, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  int64_t clusters = (g.M + g.per - 1) / g.per;
  if (TILES) clusters = std::min<int64_t>(clusters, kPerSm * clusters_at_once(kParts));  // they look for their tokens
  cfg.gridDim = dim3(unsigned(clusters * kParts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {kParts, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() || TILES ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, lora_token_kernel<XB, YB, TILES>, g);
}
template <bool XB, bool YB>
cudaError_t launch_tokens(bool tiles, const Args& g, cudaStream_t s) {
  return tiles ? launch_tokens<XB, YB, true>(g, s) : launch_tokens<XB, YB, false>(g, s);
}

}  // namespace

cudaError_t launch_lora_add(const void* x, bl_dtype xt, const int32_t* adapter, const uint16_t* a, const uint16_t* b,
                            const float* scale, const void* base, void* y, bl_dtype yt, int64_t M, int64_t N,
                            int64_t K, int64_t adapters, int rank, cudaStream_t s) {
  // A cluster per token while that is at most a few per SM; beyond, per four.
  const int per = M <= kOnePerCluster ? 1 : kGroup;
  if ((M + per - 1) / per > 0x7fffffff / kParts) return cudaErrorInvalidConfiguration;
  Args g{x, adapter, a, b, scale, base, y, dev_error_ptr(), M, N, K, adapters, rank, per};
  bool tiles = false;
  // Up to 256 tokens may be as many requests, whose tiles would be left to this kernel after a launch of the
  // other for nothing; which it is stands in device memory.  2560 -> 6912, scattered alone / with the tiles, us, rank
  // 16, 64, 128: 64 tokens of 40 runs 8 / 19, 32 / 51, 57 / 87; 256 tokens of 256 runs 25 / 43, 98 / 137, 190 / 249.
  // The price is paid by few runs in few tokens: 64 tokens of one run 11 / 11, 36 / 13, 66 / 16; 256 tokens of three
  // 17 / 13, 44 / 15, 76 / 20.  Beyond, three runs: 257 tokens, 264 -> 264, rank 8 9 / 11; 2560 -> 2560, rank 24
  // 15 / 13; 1024 tokens 25 / 11, 44 / 15.
  if (M >= kTileTokens) {
    const cudaError_t e = launch_lora_tile(x, xt, adapter, a, b, scale, base, y, yt, M, N, K, adapters, rank, s);
    if (e != cudaSuccess && e != cudaErrorNotSupported) return e;
    tiles = e == cudaSuccess;
  }
  const bool xb = xt == BL_BF16, yb = yt == BL_BF16;
  if (xb) return yb ? launch_tokens<true, true>(tiles, g, s) : launch_tokens<true, false>(tiles, g, s);
  return yb ? launch_tokens<false, true>(tiles, g, s) : launch_tokens<false, false>(tiles, g, s);
}

}  // namespace bl
