// Shared by the kernels around the paged key-value cache.
#pragma once
#include <cstdint>
#include <utility>
#include <cuda_runtime.h>

namespace bl {

// The request r with start[r] <= i < start[r + 1] (start rises; i < start[R]).
__device__ __forceinline__ int64_t request_of_token(const int32_t* start, int64_t R, int i) {
  int64_t lo = 0, hi = R;  // start[lo] <= i < start[hi]
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (start[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The rows of request r among M: start's values brought into range.
struct Rows {
  int first, n;
  bool bad;
};
__device__ __forceinline__ Rows rows_of(const int32_t* start, int64_t r, int64_t M) {
  const int a = start[r], b = start[r + 1];
  const int first = int(max(int64_t(0), min(int64_t(a), M)));
  const int end = int(max(int64_t(first), min(int64_t(b), M)));
  return {first, end - first, first != a || end != b};
}

// launch() with clusters of C CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned C, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                           bool pdl, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {C, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace bl
