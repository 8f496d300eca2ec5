// Low-rank adapters of many requests beside a shared product:
//   y[m,n] = base[m,n] + scale[a] * sum_r B[a,n,r] (sum_k A[a,r,k] x[m,k]),
// a = adapter[m], negative for none.
#include "act_quant.cuh"
#include "bl_internal.h"
#include "lora.cuh"

namespace bl {
namespace {

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
  bool tiles;  // tiles of few runs are another kernel's
};

// One CTA per token: a warp forms each of the R inner products with A's rows,
// then a thread each output.
template <bool XB, bool YB>
__global__ void __launch_bounds__(256) lora_token_kernel(const Args g) {
  __shared__ float low[128];
  const int64_t m = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  if (g.tiles) {  // the tile's runs
    const int64_t t = m / kTile * kTile + threadIdx.x;
    const bool start = threadIdx.x < kTile && t < g.M &&
                       (threadIdx.x == 0 || adapter_of(g.adapter, t, g.L) != adapter_of(g.adapter, t - 1, g.L));
    if (__syncthreads_count(start) <= kTileRuns) return;
  }
  int64_t l = g.adapter[m];
  if (l >= g.L) {
    if (threadIdx.x == 0 && g.err) atomicOr(g.err, BL_DEVERR_RANGE);
    l = -1;
  }
  if (l >= 0) {
    for (int r = warp; r < g.R; r += blockDim.x / 32) {
      float acc = 0.f;
      for (int64_t i = lane; i < g.K / 8; i += 32) {
        float xv[8], av[8];
        load8<XB>(g.x, m * (g.K / 8) + i, xv);
        load8<true>(g.a, (l * g.R + r) * (g.K / 8) + i, av);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc = fmaf(xv[j], av[j], acc);
      }
      acc = warp_sum(acc);
      if (lane == 0) low[r] = acc * g.scale[l];
    }
  }
  __syncthreads();
  for (int64_t n = threadIdx.x; n < g.N; n += blockDim.x) {
    const int64_t i = m * g.N + n;
    float acc = 0.f;
    if (l >= 0)
      for (int r = 0; r < g.R; r += 8) {
        float bv[8];
        load8<true>(g.b, ((l * g.N + n) * g.R + r) / 8, bv);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc = fmaf(bv[j], low[r + j], acc);
      }
    if (YB)
      reinterpret_cast<uint16_t*>(g.y)[i] =
          f32_to_bf16_bits_rn(bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(g.base)[i]) + acc);
    else
      reinterpret_cast<float*>(g.y)[i] = reinterpret_cast<const float*>(g.base)[i] + acc;
  }
  pdl_launch_dependents();
}

}  // namespace

cudaError_t launch_lora_add(const void* x, bl_dtype xt, const int32_t* adapter, const uint16_t* a, const uint16_t* b,
                            const float* scale, const void* base, void* y, bl_dtype yt, int64_t M, int64_t N,
                            int64_t K, int64_t adapters, int rank, cudaStream_t s) {
  Args g{x, adapter, a, b, scale, base, y, dev_error_ptr(), M, N, K, adapters, rank, false};
  const bool pdl = overlap_enabled();
  if (xt == BL_BF16 && M > 32) {
    const cudaError_t e = launch_lora_tile(x, adapter, a, b, scale, base, y, yt, M, N, K, adapters, rank, s);
    if (e != cudaSuccess && e != cudaErrorNotSupported) return e;
    g.tiles = e == cudaSuccess;
  }
  const dim3 grid{unsigned(M)}, block{256};
  if (xt == BL_BF16 && yt == BL_BF16) return launch(lora_token_kernel<true, true>, grid, block, 0, s, pdl, g);
  if (xt == BL_BF16) return launch(lora_token_kernel<true, false>, grid, block, 0, s, pdl, g);
  if (yt == BL_BF16) return launch(lora_token_kernel<false, true>, grid, block, 0, s, pdl, g);
  return launch(lora_token_kernel<false, false>, grid, block, 0, s, pdl, g);
}

}  // namespace bl
