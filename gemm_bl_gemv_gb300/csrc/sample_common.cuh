// Pieces shared by the sampling kernels (bf16 and fp32 logits).
#pragma once
#include <algorithm>

#include "bl_internal.h"
#include "sample_weight.cuh"

namespace bl {

using u64 = unsigned long long;

struct SampleArgs {
  const void* logits;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int64_t M, V;
  int32_t* token;
  float* prob;
  int chunk;  // logits of a CTA
  bool copy;  // fp32: a chunk is kept in shared memory
};

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum of the lanes up to this one.
template <class T>
__device__ __forceinline__ T warp_scan(T v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T w = __shfl_up_sync(0xffffffffu, v, o);
    if (int(threadIdx.x & 31) >= o) v += w;
  }
  return v;
}

// All threads of the cluster; the cluster barrier wants converged warps.
template <int C>
__device__ __forceinline__ void sync_cluster() {
  if (C == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    cluster_sync();
  }
}

// `grid` CTAs of `threads` in clusters of C.
template <int C>
cudaError_t launch_clusters(void (*kernel)(const SampleArgs), int64_t grid, int threads, int smem, cudaStream_t s,
                            const SampleArgs& g) {
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t e = raise_smem_cap(kernel, dev, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (C > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim = {C, 1, 1};
    ++n;
  }
  if (overlap_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, g);
}

// The number of CTAs of a row: cost(c) is the time of a row in c CTAs.
template <class F>
int ctas_per_row(int64_t M, F cost) {
  int best = 1;
  double least = 0;
  for (int c = 1; c <= 8; c *= 2) {
    const int64_t at_once = clusters_at_once(c);
    const double t = double((M + at_once - 1) / at_once) * cost(c);
    if (c == 1 || t < 0.95 * least) best = c, least = t;
  }
  return best;
}

}  // namespace bl
