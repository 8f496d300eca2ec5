// One token per row of logits by temperature, top-k, top-p and min-p from a
// given uniform number.  All three filters keep a prefix of the tokens in the
// order of falling logits (ties by rising index), and the token is the place
// where the cumulative weight of that order passes a target, so everything is
// "find the place in the order where a count, or a weight, is reached".
// Weights are integers (sample_weight.cuh), so sums are exact and a histogram
// filled by atomics in any order is deterministic.
#include "bl_internal.h"
#include "sample_weight.cuh"

namespace bl {
namespace {

using u64 = unsigned long long;

struct Args {
  const void* logits;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int64_t M, V;
  int32_t* token;
  float* prob;
};

template <bool LB>
__device__ __forceinline__ float load(const void* x, int64_t i) {
  if (LB) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(x)[i]);
  return reinterpret_cast<const float*>(x)[i];
}

// A place in the order: the element of this key with `rank` others of the
// same key before it; `before` is the weight of everything before that key.
struct Place {
  uint32_t key;
  u64 rank, before, weight;
};

struct Shared {
  Exp2Table exp2;
  unsigned int count[256];
  u64 mass[256];
  float red[32];
  u64 redu[32];
  unsigned int digit;
  u64 skip_count, skip_mass;
  unsigned int scan[1024];
};

template <bool LB>
struct RowSampler {
  const Args& g;
  Shared& sh;
  int64_t base;
  float top;
  Slope slope;

  __device__ u64 block_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.redu[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < int(blockDim.x / 32); ++w) v += sh.redu[w];
    return v;
  }

  // The place where the cumulative count (by_count) or weight first exceeds
  // `goal`, by radix descent over the key's four bytes.
  __device__ Place find(bool by_count, u64 goal) {
    uint32_t prefix = 0, mask = 0;
    u64 before_count = 0, before_mass = 0;
    for (int sft = 24; sft >= 0; sft -= 8) {
      __syncthreads();
      for (int i = threadIdx.x; i < 256; i += blockDim.x) sh.count[i] = 0, sh.mass[i] = 0;
      __syncthreads();
      for (int64_t i = threadIdx.x; i < g.V; i += blockDim.x) {
        const uint32_t k = key_of_f32(load<LB>(g.logits, base + i));
        if ((k & mask) != prefix) continue;
        const int d = (k >> sft) & 255;
        atomicAdd(&sh.count[d], 1u);
        atomicAdd(&sh.mass[d], weight_of(f32_of_key(k), top, slope, sh.exp2));
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        u64 c = before_count, w = before_mass;
        int d = 255;
        for (; d > 0; --d) {
          if (by_count ? c + sh.count[d] > goal : w + sh.mass[d] > goal) break;
          c += sh.count[d];
          w += sh.mass[d];
        }
        sh.digit = d;
        sh.skip_count = c;
        sh.skip_mass = w;
      }
      __syncthreads();
      prefix |= sh.digit << sft;
      mask |= 255u << sft;
      before_count = sh.skip_count;
      before_mass = sh.skip_mass;
    }
    const u64 w = weight_of(f32_of_key(prefix), top, slope, sh.exp2);
    return Place{prefix, by_count ? goal - before_count : (w ? (goal - before_mass) / w : 0), before_mass, w};
  }
};

template <bool LB>
__global__ void __launch_bounds__(1024) sample_any_kernel(const Args g) {
  __shared__ Shared sh;
  const int64_t m = blockIdx.x;
  pdl_wait();
  fill_exp2_table(sh.exp2);
  RowSampler<LB> row{g, sh, m * g.V, -INFINITY, {}};
  float t = -INFINITY;
  for (int64_t i = threadIdx.x; i < g.V; i += blockDim.x) t = fmaxf(t, load<LB>(g.logits, row.base + i));
  t = warp_max(t);
  if ((threadIdx.x & 31) == 0) sh.red[threadIdx.x >> 5] = t;
  __syncthreads();
  for (int w = 0; w < int(blockDim.x / 32); ++w) t = fmaxf(t, sh.red[w]);
  if (t == -INFINITY) {
    if (threadIdx.x == 0) {
      g.token[m] = -1;
      if (g.prob) g.prob[m] = 0.f;
    }
    pdl_launch_dependents();
    return;
  }
  const RowFilter f = row_filter(RowValues(m, g.temperature, g.top_k, g.top_p, g.min_p, g.u), g.V);
  row.top = t + 0.f;
  row.slope = f.slope;
  Place end{0, 0, 0, 0};  // the last place that stays
  u64 kept = 0;
  bool whole = f.top_k >= g.V;
  if (whole) {
    for (int64_t i = threadIdx.x; i < g.V; i += blockDim.x)
      kept += weight_of(load<LB>(g.logits, row.base + i), row.top, row.slope, sh.exp2);
    kept = row.block_sum(kept);
  } else {
    end = row.find(true, f.top_k - 1);
    kept = end.before + (end.rank + 1) * end.weight;
  }
  if (f.top_p <= 1.f) {
    const u64 limit = mass_limit(f.top_p, kept);
    if (limit > 0 && limit <= kept) {
      end = row.find(false, limit - 1);  // the first place whose cumulative weight reaches the limit
      whole = false;
    } else if (limit == 0) {
      end = row.find(true, 0);
      whole = false;
    }
    if (!whole) kept = end.before + (end.rank + 1) * end.weight;
  }
  if (f.min_w > 0 && (whole || end.weight < f.min_w)) {
    kept = 0;
    for (int64_t i = threadIdx.x; i < g.V; i += blockDim.x) {
      const u64 w = weight_of(load<LB>(g.logits, row.base + i), row.top, row.slope, sh.exp2);
      if (w >= f.min_w) kept += w;
    }
    kept = row.block_sum(kept);
  }
  const Place at = row.find(false, mass_target(f.u, kept));
  // the element of that key with at.rank equal ones before it, in the order of the indices
  const int64_t per = (g.V + blockDim.x - 1) / blockDim.x;
  const int64_t lo = per * threadIdx.x, hi = lo + per < g.V ? lo + per : g.V;
  unsigned int mine = 0;
  for (int64_t i = lo; i < hi; ++i) mine += key_of_f32(load<LB>(g.logits, row.base + i)) == at.key;
  sh.scan[threadIdx.x] = mine;
  __syncthreads();
  u64 skip = 0;
  for (int i = 0; i < int(threadIdx.x); ++i) skip += sh.scan[i];
  if (skip <= at.rank && at.rank < skip + mine) {
    for (int64_t i = lo; i < hi; ++i) {
      if (key_of_f32(load<LB>(g.logits, row.base + i)) != at.key) continue;
      if (skip++ == at.rank) {
        g.token[m] = int32_t(i);
        if (g.prob) g.prob[m] = share_of(f32_of_key(at.key), row.top, row.slope, sh.exp2, kept);
        break;
      }
    }
  }
  pdl_launch_dependents();
}

}  // namespace

cudaError_t launch_sample(const void* logits, bl_dtype lt, const float* temperature, const int32_t* top_k,
                          const float* top_p, const float* min_p, const float* u, int64_t M, int64_t V,
                          int32_t* token, float* prob, cudaStream_t s) {
  const Args g{logits, temperature, top_p, min_p, u, top_k, M, V, token, prob};
  const bool pdl = overlap_enabled();
  const dim3 grid{unsigned(M)}, block{1024};
  if (lt == BL_BF16)
    return launch_sample_bf16(static_cast<const uint16_t*>(logits), temperature, top_k, top_p, min_p, u, M, V, token,
                              prob, s);
  return launch(sample_any_kernel<false>, grid, block, 0, s, pdl, g);
}

}  // namespace bl
