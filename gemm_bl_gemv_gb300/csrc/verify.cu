// Verification of drafted tokens (bl_verify).  With p and q the softmax of the
// target's and the draft's logits / temperature, a request's drafts are accepted
// from the left while u q(x) < p(x); then one token is drawn in the order of the
// vocabulary, from max(p - q, 0) where a draft was refused, from p after the last.
//
// The first kernel forms maximum and mass of all rows that have a draft, each row cut
// into stretches so that few rows fill the GPU; for the tests of acceptance, which are
// comparisons of two numbers, fp32 will do.  The second kernel takes a cluster per
// request: it joins the stretches, finds the row where the request stops, and draws
// from that row.  There the sums' borders between neighbouring tokens count, so the
// weights are integers (sample_weight.cuh) and their sums exact; for max(p - q, 0)
// both are brought to units of 2^-60 by an integer reciprocal of their mass.
//
// Bound: HBM and exponentials in the first kernel, instruction issue in the second.
#include <cfloat>

#include "bl_device.cuh"
#include "bl_internal.h"
#include "paged.cuh"
#include "sample_common.cuh"

namespace bl {
namespace {

constexpr int kMassThreads = 256;
constexpr int kMostStretches = 16;
constexpr int kC = 8;  // CTAs of a request
constexpr int kThreads = 512, kWarps = kThreads / 32;

struct Args {
  const void *logits, *drafts;
  const int32_t *token, *start;
  const float *temperature, *u, *u_sample;
  int64_t M, R, V;
  int32_t *accepted, *next;
  float2* part;  // [row][target, draft][stretch]: maximum, mass
  int stretches;
  unsigned int* err;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool XB>
__device__ __forceinline__ float logit(const void* x, int64_t i) {
  return XB ? bf16_bits_to_f32(static_cast<const uint16_t*>(x)[i]) : static_cast<const float*>(x)[i];
}

// log2(e) / temperature; negative: greedy, only the maxima have weight.
__device__ __forceinline__ float rate_of(const float* temperature, int64_t r) {
  const float t = temperature ? temperature[r] : 1.f;
  return t >= kGreedyBelow ? 1.44269504f / t : -1.f;
}

// Weight of l beside a maximum (which has 1), NaN as -inf.
__device__ __forceinline__ float weight(float l, float top, float rate) {
  return rate < 0.f ? float(l == top) : l == top ? 1.f : exp2_fast(fmaxf((l - top) * rate, -200.f));
}

// Maximum and mass of the logits of two sets.
__device__ __forceinline__ float2 join(float2 a, float2 b, float rate) {
  const float top = fmaxf(a.x, b.x);
  return make_float2(top, a.y * weight(a.x, top, rate) + b.y * weight(b.x, top, rate));
}

template <bool XB>
__global__ void __launch_bounds__(kMassThreads) verify_mass_kernel(const Args a) {
  __shared__ int64_t found;
  __shared__ float2 red[kMassThreads / 32];
  const int mats = a.drafts ? 2 : 1;
  const int64_t row = blockIdx.x / (a.stretches * mats);
  const int mat = int(blockIdx.x / a.stretches % mats), stretch = int(blockIdx.x % a.stretches);
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  pdl_wait();
  // the request that has this row and a draft behind it
  for (int64_t r = threadIdx.x; r < a.R; r += kMassThreads) {
    const Rows q = rows_of(a.start, r, a.M);
    if (row >= q.first && row + 1 < int64_t(q.first) + q.n) found = r;
  }
  __syncthreads();
  if (found >= 0) {
    const float rate = rate_of(a.temperature, found);
    const void* x = mat ? a.drafts : a.logits;
    const int64_t base = row * a.V, from = a.V * stretch / a.stretches, to = a.V * (stretch + 1) / a.stretches;
    float2 s = {-FLT_MAX, 0.f};
    for (int64_t i = from + threadIdx.x; i < to; i += kMassThreads) s = join(s, {logit<XB>(x, base + i), 1.f}, rate);
    for (int o = 16; o > 0; o >>= 1)
      s = join(s, {__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)}, rate);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kMassThreads / 32; ++w) s = join(s, red[w], rate);
      a.part[(row * 2 + mat) * a.stretches + stretch] = s;
    }
  }
  pdl_launch_dependents();
}

// A mass in [2^44, 2^63] (0: none) as a 64-bit reciprocal: share(w) = w / mass in units of 2^-60.
struct Reciprocal {
  u64 r;
  int shift;
  __device__ __forceinline__ void set(u64 mass) {
    const int s = mass ? __clzll(mass) : 0;  // 0..19
    r = mass ? u64((((unsigned __int128)1 << 127) - 1) / (mass << s)) : 0;
    shift = 22 - s;
  }
  __device__ __forceinline__ u64 share(u64 w) const { return __umul64hi(w << 19, r) >> shift; }
};

// What a CTA shows the others of its cluster.
struct Shown {
  int first, n, stop;  // rank 0's: the request's rows, the draft that is refused (or how many there are)
  float top[2];
  u64 mass[2], rest[2];
};

struct __align__(16) Shared {
  Exp2Table exp2;
  Shown shown;
  Reciprocal share[2];
  u64 warps[kWarps];
  float redf[kWarps];
};

// Sum over the CTA's threads, in all of them.
__device__ __forceinline__ u64 cta_sum(u64 v, u64* warps) {
  v = warp_sum_u64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 s = 0;
  for (int w = 0; w < kWarps; ++w) s += warps[w];
  return s;
}

template <bool XB>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const Args a) {
  __shared__ Shared sh;
  const int64_t r = blockIdx.x / kC;
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  fill_exp2_table(sh.exp2);
  pdl_wait();
  const float t = a.temperature ? a.temperature[r] : 1.f;
  const float rate = rate_of(a.temperature, r);
  const Rows rows = rows_of(a.start, r, a.M);
  const int drafts = max(rows.n - 1, 0);
  bool bad = rows.bad;
  if (tid == 0) sh.shown.first = rows.first, sh.shown.n = rows.n, sh.shown.stop = drafts;
  __syncthreads();

  // the first draft that is refused
  auto mass_of = [&](int64_t row, int mat) {
    const float2* p = a.part + (row * 2 + mat) * a.stretches;
    float2 s = p[0];
    for (int i = 1; i < a.stretches; ++i) s = join(s, p[i], rate);
    return s;
  };
  for (int j = tid; rank == 0 && j < drafts; j += kThreads) {
    const int64_t row = int64_t(rows.first) + j;
    const int x = a.token[row + 1];
    double px = 0, qx = 1;
    if (x < 0 || x >= a.V) {
      bad = true;
    } else {
      const float2 p = mass_of(row, 0);
      if (p.y > 0.f) px = double(weight(logit<XB>(a.logits, row * a.V + x), p.x, rate)) / double(p.y);
      if (a.drafts) {
        const float2 q = mass_of(row, 1);
        qx = q.y > 0.f ? double(weight(logit<XB>(a.drafts, row * a.V + x), q.x, rate)) / double(q.y) : 0.0;
      }
    }
    const float u = a.u[row];
    if (!(double(u > 0.f ? fminf(u, 0.99999994f) : 0.f) * qx < px)) atomicMin(&sh.shown.stop, j);
  }
  sync_cluster<kC>();
  const Shown* first = peer(&sh.shown, 0);  // one CTA decides for all
  const int n = first->n, stop = first->stop;
  const bool refused = stop < n - 1;
  const int64_t row = int64_t(first->first) + stop, base = row * a.V;
  const int from = int(a.V * rank / kC), to = int(a.V * (rank + 1) / kC);
  // this warp's part of the CTA's
  const int wfrom = from + int(int64_t(to - from) * warp / kWarps), wto = from + int(int64_t(to - from) * (warp + 1) / kWarps);
  const bool both = refused && a.drafts;
  const Slope slope = slope_of(t);

  if (n > 0) {
    float top[2] = {-INFINITY, -INFINITY};
    for (int m = 0; m < 2; ++m) {
      if (m == 1 && !both) break;
      const void* x = m ? a.drafts : a.logits;
      float v = -INFINITY;
      for (int i = from + tid; i < to; i += kThreads) v = fmaxf(v, logit<XB>(x, base + i));
      v = warp_max(v);
      __syncthreads();
      if (lane == 0) sh.redf[warp] = v;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) v = fmaxf(v, sh.redf[w]);
      if (tid == 0) sh.shown.top[m] = v;
    }
    sync_cluster<kC>();
    for (int m = 0; m < 2; ++m)
      if (m == 0 || both)
        for (uint32_t c = 0; c < kC; ++c) top[m] = fmaxf(top[m], *peer(&sh.shown.top[m], c));
    auto weight_at = [&](int m, int i) {
      return top[m] == -INFINITY ? 0ull : weight_of(logit<XB>(m ? a.drafts : a.logits, base + i), top[m], slope, sh.exp2);
    };
    u64 mass[2] = {0, 0};
    if (both) {
      for (int m = 0; m < 2; ++m) {
        u64 s = 0;
        for (int i = from + tid; i < to; i += kThreads) s += weight_at(m, i);
        s = cta_sum(s, sh.warps);
        if (tid == 0) sh.shown.mass[m] = s;
      }
      sync_cluster<kC>();
      for (int m = 0; m < 2; ++m)
        for (uint32_t c = 0; c < kC; ++c) mass[m] += *peer(&sh.shown.mass[m], c);
    }
    if (tid < 2) sh.share[tid].set(mass[tid]);
    __syncthreads();
    const int x = refused ? a.token[row + 1] : -1;
    const Reciprocal rp = sh.share[0], rq = sh.share[1];
    // attempt 0: what p has over q; 1: p, where nothing is left
    auto rest_at = [&](int attempt, int i) {
      const u64 w = weight_at(0, i);
      if (attempt == 1 || !refused) return w;
      if (!both) return i == x ? 0ull : w;
      const u64 p = rp.share(w), q = rq.share(weight_at(1, i));
      return p > q ? p - q : 0ull;
    };
    for (int attempt = 0; attempt < 2; ++attempt) {
      u64 s = 0;
      for (int i = wfrom + lane; i < wto; i += 32) s += rest_at(attempt, i);
      s = warp_sum_u64(s);
      __syncthreads();
      if (lane == 0) sh.warps[warp] = s;
      __syncthreads();
      if (tid == 0) {
        u64 all = 0;
        for (int w = 0; w < kWarps; ++w) all += sh.warps[w];
        sh.shown.rest[attempt] = all;
      }
      sync_cluster<kC>();
      u64 all = 0, before = 0, mine = 0;
      for (uint32_t c = 0; c < kC; ++c) {
        const u64 v = *peer(&sh.shown.rest[attempt], c);
        if (c < rank) before += v;
        if (c == rank) mine = v;
        all += v;
      }
      if (all == 0) {
        if (attempt == 0 && refused) continue;
        if (rank == 0 && tid == 0) a.next[r] = -1;
        break;
      }
      const float us = a.u_sample[r];
      const u64 target = mass_target(us > 0.f ? fminf(us, 0.99999994f) : 0.f, all);
      if (before <= target && target < before + mine) {  // in this CTA's part
        u64 at = before;
        int w = 0;
        while (at + sh.warps[w] <= target) at += sh.warps[w++];
        const int f = from + int(int64_t(to - from) * w / kWarps), e = from + int(int64_t(to - from) * (w + 1) / kWarps);
        __syncthreads();  // sh.warps has been read
        for (int i0 = f; i0 < e; i0 += kThreads) {
          const u64 v = i0 + tid < e ? rest_at(attempt, i0 + tid) : 0ull;
          const u64 through = warp_scan(v);
          if (lane == 31) sh.warps[warp] = through;
          __syncthreads();
          u64 b = at;
          for (int k = 0; k < kWarps; ++k) {
            if (k < warp) b += sh.warps[k];
            at += sh.warps[k];
          }
          b += through - v;
          if (b <= target && target < b + v) a.next[r] = i0 + tid;
          __syncthreads();
        }
      }
      break;
    }
  } else if (rank == 0 && tid == 0) {
    a.next[r] = -1;
  }
  if (rank == 0 && tid == 0) a.accepted[r] = stop;
  if (__syncthreads_or(bad) && rank == 0 && tid == 0) atomicOr(a.err, BL_DEVERR_RANGE);
  sync_cluster<kC>();  // what this CTA shows has been read
  pdl_launch_dependents();
}

}  // namespace

size_t verify_workspace(int64_t M) { return size_t(M) * 2 * kMostStretches * sizeof(float2); }

cudaError_t launch_verify(const void* logits, const void* draft_logits, bl_dtype lt, const int32_t* token,
                          const int32_t* start, const float* temperature, const float* u, const float* u_sample, int64_t M,
                          int64_t R, int64_t V, int32_t* accepted, int32_t* next, void* ws, cudaStream_t s) {
  unsigned int* err = dev_error_ptr();
  if (!err) return cudaErrorUnknown;
  Args a{logits, draft_logits, token, start, temperature, u, u_sample, M, R, V, accepted, next, static_cast<float2*>(ws), 1, err};
  const int mats = draft_logits ? 2 : 1;
  a.stretches = int(std::max<int64_t>(1, std::min<int64_t>({kMostStretches, 8 * sm_count() / (M * mats), V / 4096})));
  const bool pdl = overlap_enabled();
  const dim3 grid(unsigned(M * mats * a.stretches));
  const cudaError_t e = lt == BL_BF16 ? launch(verify_mass_kernel<true>, grid, dim3(kMassThreads), 0, s, pdl, a)
                                      : launch(verify_mass_kernel<false>, grid, dim3(kMassThreads), 0, s, pdl, a);
  if (e != cudaSuccess) return e;
  // The second kernel waits for the whole first one, so the two may overlap in either setting.
  return lt == BL_BF16 ? launch_cluster(verify_draw_kernel<true>, kC, dim3(unsigned(R * kC)), dim3(kThreads), 0, s, true, a)
                       : launch_cluster(verify_draw_kernel<false>, kC, dim3(unsigned(R * kC)), dim3(kThreads), 0, s, true, a);
}

}  // namespace bl
