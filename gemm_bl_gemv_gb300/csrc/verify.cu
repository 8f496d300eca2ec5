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
// weights are integers in units of 2^-44 and their sums exact; for max(p - q, 0) both
// are brought to units of 2^-60 by an integer reciprocal of their mass.  A token's own
// weight need not be better than its stretch of the sum is wide: those below 2^-8 of the
// largest come from the hardware's exp2 (2^-22, without a bias between them and the
// others: their exponent is formed from an exact offset), in 10 instructions; the few
// others from sample_weight.cuh (2^-30), in 40.
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

// f(v, i) for elements [from, to) of MATS rows at x[m] + base, shared by n threads (this is the t-th): v[m] holds the
// elements i, i + 1, ... of row m, as many as 16 bytes have, or one at the ends.  The rows' addresses are equal modulo 16
// (`wide`), or every element comes by itself.  Several loads are in flight.
template <bool XB, int MATS, class F>
__device__ __forceinline__ void each(const void* const (&x)[2], bool wide, int64_t base, int from, int to, int t, int n, F f) {
  constexpr int E = XB ? 8 : 4, kAtOnce = MATS == 1 ? 4 : 2;
  const int off = int((reinterpret_cast<uintptr_t>(x[0]) / (XB ? 2 : 4) + uint64_t(base) + uint64_t(from)) % E);
  const int body = wide ? min(to, from + (E - off) % E) : to;  // of [from, to): from here on 16-byte words
  const int words = (to - body) / E, tail = body + words * E;
  for (int i = t; i < body - from + to - tail; i += n) {
    const int at = i < body - from ? from + i : tail + i - (body - from);
    float v[MATS][1];
#pragma unroll
    for (int m = 0; m < MATS; ++m) v[m][0] = logit<XB>(x[m], base + at);
    f(v, at);
  }
  for (int w0 = t; w0 < words; w0 += kAtOnce * n) {
    uint4 raw[kAtOnce][MATS];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
      for (int m = 0; m < MATS; ++m)
        if (w0 + j * n < words)
          raw[j][m] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x[m]) + (base + body + int64_t(w0 + j * n) * E) * (XB ? 2 : 4));
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (w0 + j * n < words) {
        float v[MATS][E];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          const uint32_t u[4] = {raw[j][m].x, raw[j][m].y, raw[j][m].z, raw[j][m].w};
#pragma unroll
          for (int e = 0; e < E; ++e) v[m][e] = __uint_as_float(!XB ? u[e % 4] : e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
        }
        f(v, body + (w0 + j * n) * E);
      }
  }
}
template <int N>
struct Count {
  static constexpr int n = N;
};
template <int MATS, int N>
__device__ __forceinline__ Count<N> count_of(const float (&)[MATS][N]) {
  return {};
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
    const int from = int(a.V * stretch / a.stretches), to = int(a.V * (stretch + 1) / a.stretches);
    float2 s = {-FLT_MAX, 0.f};
    each<XB, 1>({x, x}, true, row * a.V, from, to, threadIdx.x, kMassThreads, [&](auto& v, int) {
      constexpr int N = decltype(count_of(v))::n;
      float top = s.x;
#pragma unroll
      for (int e = 0; e < N; ++e) top = fmaxf(top, v[0][e]);
      if (top > s.x) s = make_float2(top, s.y * weight(s.x, top, rate));
      if (rate < 0.f || top == INFINITY) {
#pragma unroll
        for (int e = 0; e < N; ++e) s.y += float(v[0][e] == top);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) s.y += exp2_fast(fmaxf((v[0][e] - top) * rate, -200.f));  // NaN: 0
      }
    });
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

// Weights of a row's logits beside its largest, in units of 2^-44: light ones, below 2^-8 of the largest, by the
// hardware's exp2.
struct Weights {
  float top;
  Slope slope;
  float k, rest;  // top log2(e) / T - 40 = k + rest
  bool none, few;  // no logit above -inf; greedy or an infinity, where only the largest have weight

  __device__ __forceinline__ void set(float largest, Slope s) {
    top = largest;
    slope = s;
    none = top == -INFINITY;
    few = s.hi < 0.f || top == INFINITY;
    const float p = __fmul_rn(top, s.hi);
    k = __fsub_rn(p, 40.f);
    // what the two roundings left, and the slope's lower part
    const float z = __fsub_rn(k, p);
    rest = __fsub_rn(p, __fsub_rn(k, z)) - __fadd_rn(40.f, z);
    rest += __fmaf_rn(top, s.hi, -p) + __fmul_rn(top, s.lo);
  }
  // log2 of the weight in units of 2^-40; not below 32 (or NaN) where the weight is not light
  __device__ __forceinline__ float light(float l) const {
    l = fmaxf(l, -FLT_MAX);  // NaN and -inf
    return __fmaf_rn(l, slope.hi, -k) + __fmaf_rn(l, slope.lo, -rest);
  }
  __device__ __forceinline__ u64 full(float l, const Exp2Table& t) const {
    return none ? 0ull : few ? u64(l == top) << kWeightBits : weight_of(l, top, slope, t);
  }
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

template <bool XB, int kC>  // kC: CTAs of a request
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const Args a) {
  __shared__ Shared sh;
  const int64_t r = blockIdx.x / kC;
  const int rank = kC == 1 ? 0 : int(cluster_ctarank());
  auto of = [&](auto* p, int c) { return kC == 1 ? p : peer(p, c); };  // p in CTA c's shared memory
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
  const Shown* first = of(&sh.shown, 0);  // one CTA decides for all
  const int n = first->n, stop = first->stop;
  const bool refused = stop < n - 1;
  const int64_t row = int64_t(first->first) + stop, base = row * a.V;
  const int from = int(a.V * rank / kC), to = int(a.V * (rank + 1) / kC);
  // where warp w's part of [f, e) begins
  auto part = [](int f, int e, int w) { return f + int(int64_t(e - f) * w / kWarps); };
  const bool both = refused && a.drafts;
  const Slope slope = slope_of(t);

  if (n > 0) {
    const void* const x[2] = {a.logits, both ? a.drafts : a.logits};
    const bool wide = ((reinterpret_cast<uintptr_t>(x[0]) ^ reinterpret_cast<uintptr_t>(x[1])) & 15) == 0;
    const void* const xd[2] = {x[1], x[1]};
    float top[2] = {-INFINITY, -INFINITY};
    for (int m = 0; m < 2; ++m) {
      if (m == 1 && !both) break;
      float most = -INFINITY;
      each<XB, 1>(m ? xd : x, true, base, from, to, tid, kThreads, [&](auto& v, int) {
#pragma unroll
        for (int e = 0; e < decltype(count_of(v))::n; ++e) most = fmaxf(most, v[0][e]);
      });
      most = warp_max(most);
      __syncthreads();
      if (lane == 0) sh.redf[warp] = most;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) most = fmaxf(most, sh.redf[w]);
      if (tid == 0) sh.shown.top[m] = most;
    }
    sync_cluster<kC>();
    Weights w[2];
    for (int m = 0; m < 2; ++m) {
      if (m == 0 || both)
        for (int c = 0; c < kC; ++c) top[m] = fmaxf(top[m], *of(&sh.shown.top[m], c));
      w[m].set(top[m], slope);
    }
    // The sum of the weights of 16 bytes of logits.
    auto weigh = [&](const Weights& w, const auto& l) {
      constexpr int N = sizeof(l) / sizeof(float);
      float y[N], most = -INFINITY;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        y[e] = w.light(l[e]);
        most = y[e] < 32.f ? most : 64.f;
      }
      u64 s = 0;
      if (w.few || w.none) {
        int n = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) n += l[e] == w.top;
        return w.none ? 0 : u64(n) << kWeightBits;
      }
      if (most < 32.f) {
#pragma unroll
        for (int e = 0; e < N; ++e) s += __float2uint_rn(exp2_fast(y[e]));
        return s << 4;
      }
#pragma unroll 1
      for (int e = 0; e < N; ++e) {
        float le = l[0], ye = y[0];
#pragma unroll
        for (int i = 1; i < N; ++i) le = e == i ? l[i] : le, ye = e == i ? y[i] : ye;
        s += ye < 32.f ? u64(__float2uint_rn(exp2_fast(ye))) << 4 : w.full(le, sh.exp2);
      }
      return s;
    };
    u64 mass[2] = {0, 0};
    if (both) {
      for (int m = 0; m < 2; ++m) {
        u64 s = 0;
        each<XB, 1>(m ? xd : x, true, base, from, to, tid, kThreads, [&](auto& v, int) { s += weigh(w[m], v[0]); });
        s = cta_sum(s, sh.warps);
        if (tid == 0) sh.shown.mass[m] = s;
      }
      sync_cluster<kC>();
      for (int m = 0; m < 2; ++m)
        for (int c = 0; c < kC; ++c) mass[m] += *of(&sh.shown.mass[m], c);
      if (tid < 2) sh.share[tid].set(mass[tid]);
      __syncthreads();
    }
    const int drafted = refused ? a.token[row + 1] : -1;
    // light weights of p and q in units of 2^-40 of the masses
    constexpr float kOne = float(1ull << kWeightBits);
    const float fp = mass[0] ? kOne / float(mass[0]) : 0.f, fq = mass[1] ? kOne / float(mass[1]) : 0.f;
    // One token's share of what is drawn from: attempt 0: what p has over q; 1: p, where nothing is left.
    auto rest_at = [&](int attempt, float lp, float lq, int i) {
      const float yp = w[0].light(lp);
      const bool light = yp < 32.f && !w[0].few && !w[0].none;
      if (attempt == 1 || !both) {
        if (attempt == 0 && i == drafted) return u64(0);
        return light ? u64(__float2uint_rn(exp2_fast(yp))) << 4 : w[0].full(lp, sh.exp2);
      }
      const float yq = w[1].light(lq);
      const bool light_q = yq < 32.f && !w[1].few && !w[1].none;
      if (light && light_q) return u64(__float2uint_rn(__fmaf_rn(exp2_fast(yp), fp, -__fmul_rn(exp2_fast(yq), fq)))) << 20;
      const u64 p = sh.share[0].share(light ? u64(__float2uint_rn(exp2_fast(yp))) << 4 : w[0].full(lp, sh.exp2));
      const u64 q = sh.share[1].share(light_q ? u64(__float2uint_rn(exp2_fast(yq))) << 4 : w[1].full(lq, sh.exp2));
      return p > q ? p - q : u64(0);
    };
    const u64 few_only = both ? sh.share[0].share(1ull << kWeightBits) : 0, few_q = both ? sh.share[1].share(1ull << kWeightBits) : 0;
    const u64 few_both = few_only > few_q ? few_only - few_q : 0;
    // The sum of those of [f, e), by a warp.
    auto sum_of = [&](int attempt, int f, int e) {
      u64 s = 0;
      if (attempt == 1 || !both) {
        each<XB, 1>(x, true, base, f, e, lane, 32, [&](auto& v, int i) {
          constexpr int N = decltype(count_of(v))::n;
          if (attempt == 0 && drafted >= i && drafted < i + N) {
#pragma unroll 1
            for (int j = 0; j < N; ++j) s += rest_at(0, logit<XB>(x[0], base + i + j), 0.f, i + j);
          } else {
            s += weigh(w[0], v[0]);
          }
        });
      } else {
        each<XB, 2>(x, wide, base, f, e, lane, 32, [&](auto& v, int i) {
          constexpr int N = decltype(count_of(v))::n;
          float yp[N], yq[N], most = -INFINITY;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            yp[j] = w[0].light(v[0][j]);
            yq[j] = w[1].light(v[1][j]);
            most = yp[j] < 32.f && yq[j] < 32.f ? most : 64.f;
          }
          if (most < 32.f && !w[0].few && !w[0].none && !w[1].few && !w[1].none) {
            u64 t = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) t += __float2uint_rn(__fmaf_rn(exp2_fast(yp[j]), fp, -__fmul_rn(exp2_fast(yq[j]), fq)));
            s += t << 20;
          } else {
#pragma unroll 1
            for (int j = 0; j < N; ++j) s += rest_at(0, logit<XB>(x[0], base + i + j), logit<XB>(x[1], base + i + j), i + j);
          }
        });
      }
      return warp_sum_u64(s);
    };
    for (int attempt = 0; attempt < 2; ++attempt) {
      const u64 s = sum_of(attempt, part(from, to, warp), part(from, to, warp + 1));
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
      for (int c = 0; c < kC; ++c) {
        const u64 v = *of(&sh.shown.rest[attempt], c);
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
        int f = from, e = to;
        while (true) {  // the warp's part that has it, cut again while it is long
          int in = 0;
          while (at + sh.warps[in] <= target) at += sh.warps[in++];
          const int nf = part(f, e, in), ne = part(f, e, in + 1);
          f = nf;
          e = ne;
          __syncthreads();  // sh.warps has been read
          if (e - f <= 2 * kThreads) break;
          const u64 t = sum_of(attempt, part(f, e, warp), part(f, e, warp + 1));
          if (lane == 0) sh.warps[warp] = t;
          __syncthreads();
        }
        for (int i0 = f; i0 < e; i0 += kThreads) {
          const int64_t i = base + i0 + tid;
          const u64 v = i0 + tid < e ? rest_at(attempt, logit<XB>(x[0], i), logit<XB>(x[1], i), i0 + tid) : 0ull;
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

// It waits for the whole first kernel, so the two may overlap in either setting.
template <bool XB, int C>
cudaError_t launch_draw(const Args& a, cudaStream_t s) {
  return launch_cluster(verify_draw_kernel<XB, C>, C, dim3(unsigned(a.R * C)), dim3(kThreads), 0, s, true, a);
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
  const bool xb = lt == BL_BF16;
  const dim3 grid(unsigned(M * mats * a.stretches));
  const cudaError_t e = xb ? launch(verify_mass_kernel<true>, grid, dim3(kMassThreads), 0, s, pdl, a)
                           : launch(verify_mass_kernel<false>, grid, dim3(kMassThreads), 0, s, pdl, a);
  if (e != cudaSuccess) return e;
  // a row in c CTAs: some passes over its share, and the exchanges
  const int c = ctas_per_row(R, [&](int c) { return 6.0 + 4.0 * (c > 1) + double(V) / c * 1e-4; });
  if (xb) return c == 1 ? launch_draw<true, 1>(a, s) : c == 2 ? launch_draw<true, 2>(a, s) : c == 4 ? launch_draw<true, 4>(a, s) : launch_draw<true, 8>(a, s);
  return c == 1 ? launch_draw<false, 1>(a, s) : c == 2 ? launch_draw<false, 2>(a, s) : c == 4 ? launch_draw<false, 4>(a, s) : launch_draw<false, 8>(a, s);
}

}  // namespace bl
