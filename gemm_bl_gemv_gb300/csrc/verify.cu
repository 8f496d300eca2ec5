// Verification of drafted tokens (bl_verify).  With p and q the softmax of the
// target's and the draft's logits / temperature, a request's drafts are accepted
// from the left while u q(x) < p(x); then one token is drawn in the order of the
// vocabulary, from max(p - q, 0) where a draft was refused, from p after the last.
//
// The first kernel forms maximum and mass of all rows that have a draft, each row cut
// into stretches so that few rows fill the GPU; for the tests of acceptance, which are
// comparisons of two numbers, fp32 will do (a draft's own weight is formed on its own, to
// 2^-21 however unlikely it is).  The second kernel takes a cluster per
// request: it joins the stretches, finds the row where the request stops, and draws
// from that row.  There the sums' borders between neighbouring tokens count, so the
// weights are integers in units of 2^-44 and their sums exact; for max(p - q, 0) both
// are brought to units of 2^-60 by an integer reciprocal of their mass.  A token's own
// weight need not be better than its stretch of the sum is wide: those below 2^-8 of the
// largest come from the hardware's exp2 (2^-22, without a bias between them and the
// others: their exponent is formed from an exact offset), in 10 instructions; the few
// others from sample_weight.cuh (2^-30), in 40.
//
// Bound, 64 requests of one to five rows, bf16 logits of target and draft model over 248320 tokens (157 MB): the first
// kernel takes 30 us, 5.2 TB/s (HBM 57 % of its time's peak, issue 70 %); the second 41 us, of which two passes over a
// target's and a draft's row (issue, 12 instructions a pair of logits) are 25, the third of a part and the exchanges the
// rest; 128 of the 152 SMs have work.  One request with four drafts 16 us, 32 requests with fp32 logits over 100003 tokens 44 us.
// Masses from the first kernel, which are within 2^-22, would save one pass, and move the borders between tokens by 2^-22
// over what max(p - q, 0) leaves: more than an unlikely token is wide.
#include <cfloat>

#include "bl_device.cuh"
#include "bl_internal.h"
#include "paged.cuh"
#include "sample_common.cuh"

namespace bl {
namespace {

constexpr int kMassThreads = 128;  // 64 requests: 31 us; with 256 34, with 512 39
constexpr int kMostStretches = 16;
constexpr int kThreads = 1024, kWarps = kThreads / 32;  // a lane per warp in the sums over warps
constexpr int kListed = 32;
// Exponents l log2(e) / T of this size and above differ by 64 and more between neighbouring numbers (2^-24 of it), and a
// half of a step of theirs stays below the largest exponent of fp32.
constexpr float kMostExponent = 1073741824.f;
// Light weights, below 2^-8 of the largest, are floats in units of 2^-16 of it: their logarithm is below kLight; in units
// of 2^-44 and 2^-60.
constexpr float kLight = 8.f, kLightUnits = 268435456.f, kFineUnits = 17592186044416.f;
constexpr float kLeast = 1.40129846e-45f;  // the smallest number above 0

struct Args {
  const void *logits, *drafts;
  const int32_t *token, *start;
  const float *temperature, *u, *u_sample;
  int64_t M, R, V;
  int32_t *accepted, *next;
  float2* part;  // [row][target, draft][stretch]: maximum, mass
  int stretches, stretch;  // of a row, and their length
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

// Pairs of floats for the packed fp32 instructions.
using f2 = u64;
__device__ __forceinline__ f2 pack2(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 exp2_of(f2 v) {
  float x, y;
  unpack2(v, x, y);
  return pack2(exp2_fast(x), exp2_fast(y));
}

// 16 bytes of logits.
template <bool XB>
struct Word {
  static constexpr int E = XB ? 8 : 4;
  uint32_t u[4];
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + i * (XB ? 2 : 4));
    u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
  }
  __device__ __forceinline__ float at(int e) const {
    return __uint_as_float(!XB ? u[e % 4] : e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
  }
  __device__ __forceinline__ f2 pair(int k) const { return pack2(at(2 * k), at(2 * k + 1)); }
  __device__ __forceinline__ void fill() { u[0] = u[1] = u[2] = u[3] = XB ? 0xff80ff80u : 0xff800000u; }  // -inf
  // e known at run time only
  __device__ __forceinline__ float pick(int e) const {
    float v = at(0);
#pragma unroll
    for (int j = 1; j < E; ++j) v = e == j ? at(j) : v;
    return v;
  }
  // The largest; NaN if there is one.
  __device__ __forceinline__ float most() const { return most_of<1>(this); }
  template <int N>
  static __device__ __forceinline__ float most_of(const Word* w) {
    uint32_t m[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) m[2 * i] = larger(w[i].u[0], w[i].u[1]), m[2 * i + 1] = larger(w[i].u[2], w[i].u[3]);
#pragma unroll
    for (int o = N; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; ++i) m[i] = larger(m[i], m[i + o]);
    float r = __uint_as_float(m[0]);
    if (XB) asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(m[0] << 16)), "f"(__uint_as_float(m[0] & 0xffff0000u)));
    return r;
  }

 private:
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    if (XB) {
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    } else {
      float f;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
      r = __float_as_uint(f);
    }
    return r;
  }
};

// The elements [from, to) of MATS rows at x[m] + base, shared by n threads (this is the t-th): words(w, i) gets 16 bytes
// of each row, of its elements i, i + 1, ..., and one(i) the elements at the ends.  The rows' addresses are equal modulo 16
// (`wide`), or every element comes by itself.  Of one row the next words are loaded
// before the present ones are worked on; of two there are no registers for that, and other warps to wait with.
// kTogether: words(w, i) gets the thread's next kAtOnce words, n words apart, -inf behind the last.
template <bool XB, int MATS, int kAtOnce, bool kTogether = false, class One, class Words>
__device__ __forceinline__ void each(const void* x0, const void* x1, bool wide, int64_t base, int from, int to, int t, int n, One one, Words f) {
  constexpr int E = Word<XB>::E;
  const int off = int((reinterpret_cast<uintptr_t>(x0) / (XB ? 2 : 4) + uint64_t(base) + uint64_t(from)) % E);
  const int body = wide ? min(to, from + (E - off) % E) : to;  // of [from, to): from here on 16-byte words
  const int words = (to - body) / E, tail = body + words * E;
  for (int i = t; i < body - from + to - tail; i += n) one(i < body - from ? from + i : tail + i - (body - from));
  Word<XB> next[kAtOnce][MATS];
  auto load = [&](int w0) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (w0 + j * n < words) {
        next[j][0].load(x0, base + body + int64_t(w0 + j * n) * E);
        if (MATS == 2) next[j][MATS - 1].load(x1, base + body + int64_t(w0 + j * n) * E);
      } else if (kTogether) {
        next[j][0].fill();
        if (MATS == 2) next[j][MATS - 1].fill();
      }
  };
  constexpr bool kAhead = MATS == 1;
  if (kAhead) load(t);
  for (int w0 = t; w0 < words; w0 += kAtOnce * n) {
    if (!kAhead) load(w0);
    Word<XB> now[kAtOnce][MATS];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
      for (int m = 0; m < MATS; ++m) now[j][m] = next[j][m];
    if (kAhead) load(w0 + kAtOnce * n);
    if constexpr (kTogether) {
      f(now, body + w0 * E);
    } else {
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (w0 + j * n < words) f(now[j], body + (w0 + j * n) * E);
    }
  }
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

// Weight of l beside a maximum (which has 1) as m 2^e, m returned: with the exponent's whole part kept apart, an unlikely
// token's weight is as exact as a likely one's (2^-21).  0 below 2^-1000, as where only the largest have weight.
__device__ __forceinline__ float weight_apart(float l, float top, Slope c, int& e) {
  e = 0;
  if (l == top) return 1.f;
  const Pair x = exponent_of(l, top, c);
  if (c.hi < 0.f || !(x.e > -1000.f)) return 0.f;
  const float n = rintf(x.e);
  e = int(n);
  return exp2_fast(__fsub_rn(x.e, n) + x.el);
}

// Maximum and mass of the logits of two sets.
__device__ __forceinline__ float2 join(float2 a, float2 b, float rate) {
  const float top = fmaxf(a.x, b.x);
  return make_float2(top, a.y * weight(a.x, top, rate) + b.y * weight(b.x, top, rate));
}

// A mass is within 2^-17 of its value, mostly within 2^-21: the slope's error, 2^-23.4, counts up to 19 times (a token of
// 2^-z of the largest counts if there are 2^z of them, of 2^19): 2^-20; an exponent's rounding 2^-20.5; exp2 2^-22; 26
// additions behind one another 2^-19.3; the joining of threads and stretches, two roundings of up to 19, 2^-19.3.
template <bool XB>
__global__ void __launch_bounds__(kMassThreads) verify_mass_kernel(const Args a) {
  __shared__ int64_t found;
  __shared__ float2 red[kMassThreads / 32];
  const int64_t row = blockIdx.x;
  const int mat = int(blockIdx.z), stretch = int(blockIdx.y);
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  pdl_wait();
  // the request that has this row; a row of the draft's logits has to have a draft behind it
  for (int64_t r = threadIdx.x; r < a.R; r += kMassThreads) {
    const Rows q = rows_of(a.start, r, a.M);
    if (row >= q.first && row + mat < int64_t(q.first) + q.n) found = r;
  }
  __syncthreads();
  if (found >= 0) {
    const float rate = rate_of(a.temperature, found);
    const bool few = rate < 0.f;
    const void* x = mat ? a.drafts : a.logits;
    const int from = stretch * a.stretch, to = min(int(a.V), from + a.stretch);
    // The sum is in units of 2^E, E a whole number, so that l rate - E is rounded once; -inf: only the largest have
    // weight (greedy, or exponents of kMostExponent and more, where the next smaller number has 2^-64).
    float top = -INFINITY, E = -INFINITY, sum = 0.f;
    auto raise = [&](float l) {  // to a larger maximum
      top = l;
      const float next = few || !(fabsf(l * rate) < kMostExponent) ? -INFINITY : ceilf(l * rate);
      sum *= next > -INFINITY ? exp2_fast(E - next) : 0.f;
      E = next;
    };
    auto add = [&](float l) {  // NaN: nothing
      if (l > top) raise(l);
      if (!(l > -INFINITY)) return;
      sum += E > -INFINITY ? exp2_fast(__fmaf_rn(l, rate, -E)) : float(l == top);
    };
    const f2 rate2 = pack2(rate, rate);
    // Four words at a time: their largest and what hangs on it cost more than a word's weights.
    constexpr int N = 4, kPairs = Word<XB>::E / 2;
    each<XB, 1, N, true>(x, x, true, row * a.V, from, to, threadIdx.x, kMassThreads, [&](int i) { add(logit<XB>(x, row * a.V + i)); },
                         [&](const Word<XB>(&w)[N][1], int) {
                           const float most = Word<XB>::template most_of<N>(&w[0][0]);
                           if (most > top) raise(most);
                           if (most == -INFINITY) return;
                           if (most == most && E > -INFINITY && rate > 0.f) {
                             const f2 e2 = pack2(-E, -E);
                             f2 t[N];
#pragma unroll
                             for (int i = 0; i < N; ++i) t[i] = exp2_of(fma2(w[i][0].pair(0), rate2, e2));
#pragma unroll
                             for (int k = 1; k < kPairs; ++k)
#pragma unroll
                               for (int i = 0; i < N; ++i) t[i] = add2(t[i], exp2_of(fma2(w[i][0].pair(k), rate2, e2)));
                             float t0, t1;
                             unpack2(add2(add2(t[0], t[1]), add2(t[2], t[3])), t0, t1);
                             sum += t0 + t1;
                           } else if (most == most && !(E > -INFINITY)) {
#pragma unroll
                             for (int i = 0; i < N; ++i)
#pragma unroll
                               for (int e = 0; e < Word<XB>::E; ++e) sum += float(w[i][0].at(e) == top);
                           } else {
#pragma unroll 1
                             for (int i = 0; i < N; ++i)
#pragma unroll 1
                               for (int e = 0; e < Word<XB>::E; ++e) {
                                 float l = w[0][0].pick(e);
#pragma unroll
                                 for (int k = 1; k < N; ++k) l = i == k ? w[k][0].pick(e) : l;
                                 add(l);
                               }
                           }
                         });
    // to the warp's and the CTA's largest: the sums are beside their maximum from here on, as elsewhere
    if (E > -INFINITY) sum *= exp2_fast(-__fmaf_rn(top, rate, -E));
    float most = warp_max(top);
    sum = warp_sum(sum * weight(top, most, rate));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(most, sum);
    __syncthreads();
    if (threadIdx.x < kMassThreads / 32) {
      constexpr unsigned kLanes = (1u << kMassThreads / 32) - 1;
      const float2 s = red[threadIdx.x];
      most = s.x;
#pragma unroll
      for (int o = kMassThreads / 64; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kLanes, most, o));
      sum = s.y * weight(s.x, most, rate);
#pragma unroll
      for (int o = kMassThreads / 64; o > 0; o >>= 1) sum += __shfl_xor_sync(kLanes, sum, o);
      if (threadIdx.x == 0) a.part[(row * 2 + mat) * a.stretches + stretch] = make_float2(most, sum);
    }
  }
  pdl_launch_dependents();
}

// A mass in [2^43, 2^63] (0: none) as a 64-bit reciprocal: share(w) = w / mass in units of 2^-60, to 2^-61 of it.
struct Reciprocal {
  u64 r;  // 2^127 / (mass << s)
  int shift;
  __device__ __forceinline__ void set(u64 mass) {
    const int s = mass ? __clzll(mass) : 0;  // 0..20
    const u64 n = mass << s;
    shift = 22 - s;
    r = 0;
    if (n == 1ull << 63) {
      r = ~0ull;
    } else if (mass) {
      u64 x = __float2ull_rz(__fdiv_rd(1.7014117e38f, __ull2float_ru(n)));  // a little below 2^127 / n, 23 bits
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // x += x (2^127 - n x) / 2^127: 46 bits, then all; the remainder is positive
        const u64 e = (1ull << 63) - __umul64hi(n, x) - 1;
        x += __umul64hi(x, e) * 2;
      }
      r = x;
    }
  }
  __device__ __forceinline__ u64 share(u64 w) const { return __umul64hi(w << 19, r) >> shift; }
  // The same of a sum of light weights (2^61 at most) in units of 2^-60.
  __device__ __forceinline__ u64 fine(u64 w) const { return __umul64hi(w << 2, r) >> (shift - 1); }
};

// Weights of a row's logits, 2^(l log2(e) / T - E) in units of 2^-44, where E is a whole number so near to the largest
// logit's exponent that its weight is in (2^43, 2^44].  log2(e) / T = hi + lo with lo > 0 (-inf has weight 0 then).
// `apart`: from exponents of 2^15 on, whose products are rounded by 2^-10 and more (the polynomial takes 2^-6), the weights
// are formed from the difference to the largest logit, as in the sampling.
struct Weights {
  float hi, lo, E;
  float top;
  bool none, few, apart;  // no logit above -inf; only the largest have weight: greedy, an infinity, or too large exponents
  float offset;           // 16 - E
  float least;            // logits below this one have no weight (where offset is NaN: they need not be looked at)
  Slope slope;

  __device__ __forceinline__ void set(float2 stat, float temperature) {
    top = stat.x;
    none = !(stat.y > 0.f);
    const float lh = 1.44269502162933349609375f, ll = 1.92596303313e-8f;  // log2(e) = lh + ll
    hi = fmaxf(__fdiv_rd(lh, temperature), kLeast);
    lo = fmaxf(__fdiv_rn(__fadd_rn(__fmaf_rn(-hi, temperature, lh), ll), temperature), kLeast);  // lh - hi T is exact
    const float p = __fmul_rn(top, hi);
    E = ceilf(p);
    few = !(temperature >= kGreedyBelow) || !(fabsf(p) < kMostExponent);
    apart = !(fabsf(E) < 32768.f);
    offset = !few && !none && !apart ? 16.f - E : NAN;  // every weight by full()
    slope = slope_of(temperature);
    least = few ? top : apart ? __fsub_rd(top, __fdiv_ru(64.f, hi)) : -INFINITY;
  }
  // log2 of the weight in units of 2^-16, where it is below 8 (NaN where all are formed by full()): in this unit the
  // exponents of the light weights that count, 2^-8 to 2^-24, lie within +-8, where a rounding is 2^-22.
  __device__ __forceinline__ float light(float l) const { return __fmaf_rn(l, lo, __fmaf_rn(l, hi, offset)); }
  __device__ __forceinline__ u64 full(float l, const Exp2Table& t) const {
    if (none) return 0;
    if (few) return u64(l == top) << kWeightBits;
    if (apart) return weight_of(l, top, slope, t);
    const float p = __fmul_rn(l, hi);
    const float e = __fsub_rn(p, E), z = __fsub_rn(e, p);
    const float el = __fadd_rn(__fsub_rn(p, __fsub_rn(e, z)), __fsub_rn(-E, z)) + __fmaf_rn(l, lo, __fmaf_rn(l, hi, -p));
    int shift;
    const u64 w = exp2_mantissa(e, el, false, t, shift);
    return (w + ((1ull << shift) >> 1)) >> shift;
  }
};

// What a CTA shows the others of its cluster.
struct Shown {
  int first, n, stop;  // rank 0's: the request's rows, the draft that is refused (or how many there are)
  float2 stat[2];      // rank 0's: maximum and mass (fp32) of the row in the target's and the draft's logits
  u64 mass[2], rest[2];
};

struct __align__(16) Shared {
  Exp2Table exp2;
  Shown shown;
  Weights w[2];
  Reciprocal share[2];
  float ratio[2];  // p's mass over q's, which q's light weights are multiplied by, in two terms
  u64 warps[kWarps], masses[2][kWarps];
  int listed[kWarps];          // tokens of a warp's part whose weights are not light, and where they are
  int list[kWarps][kListed];
  float value[kWarps][kListed][2];  // of p's and q's logits
};

// The weight of a logit of the target's row (m = 0) or the draft's.
__device__ __noinline__ u64 weight_in(const Shared& sh, int m, float l) {
  const float y = sh.w[m].light(l);
  return y < kLight ? __float2ull_rn(kLightUnits * exp2_fast(y)) : sh.w[m].full(l, sh.exp2);
}
// What light weights leave of p - q, as a weight of p in units of 2^-16.  Where p equals q (a ratio of 1), nothing is left:
// each fma rounds once.
__device__ __forceinline__ float light_excess(const Shared& sh, float yp, float yq) {
  const float q = exp2_fast(yq);
  return fmaxf(__fmaf_rn(q, -sh.ratio[1], __fmaf_rn(q, -sh.ratio[0], exp2_fast(yp))), 0.f);
}
// What p has over q, in units of 2^-60 of their masses.
__device__ __noinline__ u64 excess(const Shared& sh, float lp, float lq) {
  const float yp = sh.w[0].light(lp), yq = sh.w[1].light(lq);
  if (yp < kLight && yq < kLight) return sh.share[0].fine(__float2ull_rn(kFineUnits * light_excess(sh, yp, yq)));
  const u64 p = sh.share[0].share(weight_in(sh, 0, lp)), q = sh.share[1].share(weight_in(sh, 1, lq));
  return p > q ? p - q : 0;
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
  if (tid < kWarps) sh.listed[tid] = 0;
  if (tid == 0) sh.shown.first = rows.first, sh.shown.n = rows.n, sh.shown.stop = drafts;
  __syncthreads();

  // Maximum and mass of a row, lanes 0..15 the target's and the others the draft's: a lane per stretch.
  auto mass_of = [&](int64_t row, bool drafts) {
    const int i = lane % kMostStretches;
    float2 s = {-INFINITY, 0.f};
    if (i < a.stretches && (lane < kMostStretches || drafts)) s = a.part[(row * 2 + lane / kMostStretches) * a.stretches + i];
#pragma unroll
    for (int o = kMostStretches / 2; o > 0; o >>= 1)
      s = join(s, {__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)}, rate);
    return s;
  };
  // the first draft that is refused: a warp per draft
  const Slope slope = slope_of(t);
  for (int j = warp; rank == 0 && j < drafts; j += kWarps) {
    const int64_t row = int64_t(rows.first) + j;
    const int x = a.token[row + 1];
    const float u = a.u[row];
    const bool mine = lane < kMostStretches || a.drafts;
    float2 s = mass_of(row, a.drafts != nullptr);
    float w = mine ? 0.f : 1.f;  // w 2^e / s.y: p in lane 0, q in lane 16
    int e = 0;
    if (x < 0 || x >= a.V) {
      bad = true;
    } else if (mine && s.y > 0.f) {
      w = weight_apart(logit<XB>(lane < kMostStretches ? a.logits : a.drafts, row * a.V + x), s.x, slope, e);
    }
    if (!mine || !(s.y > 0.f)) s.y = 1.f;
    const float wq = __shfl_sync(0xffffffffu, w, kMostStretches), mass_q = __shfl_sync(0xffffffffu, s.y, kMostStretches);
    const int eq = __shfl_sync(0xffffffffu, e, kMostStretches);
    // u q < p with both sides times both masses and 2^-e, which fp64 has the range for
    const double u_q = double(u > 0.f ? fminf(u, 0.99999994f) : 0.f) * double(wq) * double(s.y) * __hiloint2double((1023 + eq - e) << 20, 0);
    if (lane == 0 && !(u_q < double(w) * double(mass_q))) atomicMin(&sh.shown.stop, j);
  }
  __syncthreads();
  if (rank == 0 && warp == 0 && rows.n > 0) {
    const float2 s = mass_of(int64_t(rows.first) + sh.shown.stop, a.drafts && sh.shown.stop < drafts);
    if (lane % kMostStretches == 0) sh.shown.stat[lane / kMostStretches] = s;
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

  if (n > 0) {
    const void* const x[2] = {a.logits, both ? a.drafts : a.logits};
    const bool wide = ((reinterpret_cast<uintptr_t>(x[0]) ^ reinterpret_cast<uintptr_t>(x[1])) & 15) == 0;
    if (tid < 2) sh.w[tid].set(first->stat[tid], t);
    __syncthreads();
    const int drafted = refused ? a.token[row + 1] : -1;
    // Logits whose weight is not light are few and spread; one by one they would stop their warps.  They are listed, and
    // weighed after the pass, a lane each (at once where the list is full).
    auto list = [&](int i, float lp, float lq) {
      const int k = atomicAdd(&sh.listed[warp], 1);
      if (k < kListed) sh.list[warp][k] = i, sh.value[warp][k][0] = lp, sh.value[warp][k][1] = lq;
      return k < kListed;
    };
    // f(i, lp, lq) for what this warp has listed.
    auto each_listed = [&](auto f) {
      __syncwarp();
      const int n = min(sh.listed[warp], kListed);
      for (int k = lane; k < n; k += 32) f(sh.list[warp][k], sh.value[warp][k][0], sh.value[warp][k][1]);
      __syncwarp();
      if (lane == 0) sh.listed[warp] = 0;
      __syncwarp();
    };
    auto at = [&](int m, int i) { return logit<XB>(x[m], base + i); };
    // The weights of logits from i on: light ones to `sum` (fp32: a lane has few of them), in units of 2^-16, others to
    // the list or `more`.
    auto weigh_one = [&](int m, int i, u64& more) { more += weight_in(sh, m, at(m, i)); };
    auto weigh = [&](int m, const Word<XB>& l, int i, float& sum, u64& more) {
      constexpr int N = Word<XB>::E;
      const Weights& w = sh.w[m];
      if (w.light(l.most()) < kLight) {
        const f2 hi = pack2(w.hi, w.hi), lo = pack2(w.lo, w.lo), offset = pack2(w.offset, w.offset);
        f2 t = 0;
#pragma unroll
        for (int k = 0; k < N / 2; ++k) t = add2(t, exp2_of(fma2(l.pair(k), lo, fma2(l.pair(k), hi, offset))));
        float t0, t1;
        unpack2(t, t0, t1);
        sum += t0 + t1;
      } else if (!w.none && !(l.most() < w.least)) {
        unsigned heavy = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float y = w.light(l.at(e));
          if (y < kLight)
            sum += exp2_fast(y);
          else
            heavy |= unsigned(l.at(e) > -INFINITY && !(l.at(e) < w.least)) << e;  // -inf and NaN have no weight
        }
        for (; heavy; heavy &= heavy - 1) {
          const int e = __ffs(heavy) - 1;
          const float le = l.pick(e);
          if (!list(i + e, le, le)) more += weight_in(sh, m, le);
        }
      }
    };
    const int wfrom = part(from, to, warp), wto = part(from, to, warp + 1);
    u64 mass[2] = {0, 0};
    if (both) {
      float sum[2] = {0.f, 0.f};
      // (q's entries in the list: negative)
      each<XB, 2, 1>(x[0], x[1], wide, base, wfrom, wto, lane, 32,
                     [&](int i) {
                       weigh_one(0, i, mass[0]);
                       weigh_one(1, i, mass[1]);
                     },
                     [&](const Word<XB>(&v)[2], int i) {
                       weigh(0, v[0], i, sum[0], mass[0]);
                       weigh(1, v[1], -1 - i - (Word<XB>::E - 1), sum[1], mass[1]);
                     });
      each_listed([&](int i, float l, float) {
        const u64 w = weight_in(sh, i < 0, l);
        mass[0] += i < 0 ? 0 : w;
        mass[1] += i < 0 ? w : 0;
      });
      for (int m = 0; m < 2; ++m) {
        mass[m] = warp_sum_u64(mass[m] + __float2ull_rn(kLightUnits * sum[m]));
        if (lane == 0) sh.masses[m][warp] = mass[m];
      }
      __syncthreads();
      if (warp < 2) {
        const u64 s = warp_sum_u64(sh.masses[warp][lane]);
        if (lane == 0) sh.shown.mass[warp] = s;
      }
      sync_cluster<kC>();
      if (warp == 0) {
        u64 s = 0;
        if (lane < 2) {
          for (int c = 0; c < kC; ++c) s += *of(&sh.shown.mass[lane], c);
          sh.share[lane].set(s);
        }
        const u64 of_q = __shfl_sync(0xffffffffu, s, 1);
        if (lane == 0) {
          const double ratio = of_q ? double(s) / double(of_q) : 0.0;
          sh.ratio[0] = float(ratio);
          sh.ratio[1] = float(ratio - double(sh.ratio[0]));
        }
      }
      __syncthreads();
    }
    // One token's share of what is drawn from: attempt 0: what p has over q, in units of 2^-60 of the mass, or p without
    // the draft; 1: p, where nothing is left.
    auto rest_at = [&](int attempt, int i, float lp, float lq) {
      if (attempt == 0 && both) return excess(sh, lp, lq);
      return attempt == 0 && i == drafted ? u64(0) : weight_in(sh, 0, lp);
    };
    // The sum of those of [f, e), by a warp.
    auto sum_of = [&](int attempt, int f, int e) {
      u64 more = 0;
      float sum = 0.f;
      const bool p_only = attempt == 1 || !both;
      if (p_only) {
        each<XB, 1, 2>(x[0], x[0], true, base, f, e, lane, 32, [&](int i) { more += rest_at(attempt, i, at(0, i), 0.f); },
                       [&](const Word<XB>(&v)[1], int i) {
                         if (attempt == 0 && drafted >= i && drafted < i + Word<XB>::E) {
#pragma unroll 1
                           for (int j = 0; j < Word<XB>::E; ++j) more += rest_at(0, i + j, v[0].pick(j), 0.f);
                         } else {
                           weigh(0, v[0], i, sum, more);
                         }
                       });
      } else {
        const Weights &wp = sh.w[0], &wq = sh.w[1];
        each<XB, 2, 1>(x[0], x[1], wide, base, f, e, lane, 32, [&](int i) { more += excess(sh, at(0, i), at(1, i)); },
                       [&](const Word<XB>(&v)[2], int i) {
                         constexpr int N = Word<XB>::E;
                         if (wp.light(v[0].most()) < kLight && wq.light(v[1].most()) < kLight) {
                           const f2 hp = pack2(wp.hi, wp.hi), lp = pack2(wp.lo, wp.lo), op = pack2(wp.offset, wp.offset);
                           const f2 hq = pack2(wq.hi, wq.hi), lq = pack2(wq.lo, wq.lo), oq = pack2(wq.offset, wq.offset);
                           const f2 r0 = pack2(-sh.ratio[0], -sh.ratio[0]), r1 = pack2(-sh.ratio[1], -sh.ratio[1]);
                           f2 t = 0;
#pragma unroll
                           for (int k = 0; k < N / 2; ++k) {
                             const f2 ep = exp2_of(fma2(v[0].pair(k), lp, fma2(v[0].pair(k), hp, op)));
                             const f2 eq = exp2_of(fma2(v[1].pair(k), lq, fma2(v[1].pair(k), hq, oq)));
                             float d0, d1;
                             unpack2(fma2(eq, r1, fma2(eq, r0, ep)), d0, d1);  // light_excess
                             t = add2(t, pack2(fmaxf(d0, 0.f), fmaxf(d1, 0.f)));
                           }
                           float t0, t1;
                           unpack2(t, t0, t1);
                           sum += t0 + t1;
                         } else if (!wp.none && !(v[0].most() < wp.least)) {
                           unsigned heavy = 0;
#pragma unroll
                           for (int j = 0; j < N; ++j) {
                             const float l0 = v[0].at(j), yp = wp.light(l0), yq = wq.light(v[1].at(j));
                             if (yp < kLight && yq < kLight)
                               sum += light_excess(sh, yp, yq);
                             else
                               heavy |= unsigned(l0 > -INFINITY && !(l0 < wp.least)) << j;  // p has none otherwise
                           }
                           for (; heavy; heavy &= heavy - 1) {
                             const int j = __ffs(heavy) - 1;
                             const float l0 = v[0].pick(j), l1 = v[1].pick(j);
                             if (!list(i + j, l0, l1)) more += excess(sh, l0, l1);
                           }
                         }
                       });
      }
      each_listed([&](int i, float lp, float lq) { more += rest_at(attempt, i, lp, lq); });
      return warp_sum_u64(more + (p_only ? __float2ull_rn(kLightUnits * sum) : sh.share[0].fine(__float2ull_rn(kFineUnits * sum))));
    };
    for (int attempt = 0; attempt < 2; ++attempt) {
      const u64 s = sum_of(attempt, wfrom, wto);
      __syncthreads();
      if (lane == 0) sh.warps[warp] = s;
      __syncthreads();
      if (warp == 0) {
        const u64 all = warp_sum_u64(sh.warps[lane]);
        if (lane == 0) sh.shown.rest[attempt] = all;
      }
      sync_cluster<kC>();
      const u64 theirs = lane < kC ? *of(&sh.shown.rest[attempt], lane) : 0;
      const u64 up_to = warp_scan(theirs);
      const u64 all = __shfl_sync(0xffffffffu, up_to, 31), through_mine = __shfl_sync(0xffffffffu, up_to, rank);
      const u64 before = through_mine - __shfl_sync(0xffffffffu, theirs, rank);
      if (all == 0) {
        if (attempt == 0 && refused) continue;
        if (rank == 0 && tid == 0) a.next[r] = -1;
        break;
      }
      const float us = a.u_sample[r];
      const u64 target = mass_target(us > 0.f ? fminf(us, 0.99999994f) : 0.f, all);
      if (before <= target && target < through_mine) {  // in this CTA's part
        u64 through_parts = before;
        int f = from, e = to;
        while (true) {  // the warp's part that has it, cut again while it is long
          const u64 v = sh.warps[lane], through = warp_scan(v);
          const unsigned live = __ballot_sync(0xffffffffu, v != 0), past = __ballot_sync(0xffffffffu, through_parts + through > target);
          // A lane rounds its sum once, so a part may have one where none of those that it is cut into does: then it is
          // looked through as it is.
          if (live) {
            const int in = past ? __ffs(past) - 1 : 31 - __clz(live);  // the last that has any, where the sums end early
            through_parts += __shfl_sync(0xffffffffu, through - v, in);
            const int nf = part(f, e, in), ne = part(f, e, in + 1);
            f = nf;
            e = ne;
          }
          __syncthreads();  // sh.warps has been read
          if (!live || e - f <= 2 * kThreads) break;
          const u64 t = sum_of(attempt, part(f, e, warp), part(f, e, warp + 1));
          if (lane == 0) sh.warps[warp] = t;
          __syncthreads();
        }
        // The part's sum was formed in another order than the tokens' own shares are: where these end before the
        // target, the last token that has one is taken, and where they are below their unit the token that has most.
        auto light_share = [&](int i, float lp, float lq) {  // unrounded; of a weight that is not light the share is whole
          const float yp = sh.w[0].light(lp), yq = sh.w[1].light(lq);
          if (!(yp < kLight)) return 0.f;
          if (attempt == 0 && both) return yq < kLight ? light_excess(sh, yp, yq) : 0.f;
          return attempt == 0 && i == drafted ? 0.f : exp2_fast(yp);
        };
        u64 best = 0;  // (whether it has a share, its light one) over the token
        for (int i0 = f; i0 < e; i0 += kThreads) {
          const int i = i0 + tid;
          const float l = i < e ? at(0, i) : -INFINITY, lq = i < e ? at(1, i) : -INFINITY;
          const u64 v = i < e ? rest_at(attempt, i, l, lq) : 0ull;
          const u64 through = warp_scan(v);
          if (lane == 31) sh.warps[warp] = through;
          __syncthreads();
          const u64 w = sh.warps[lane], through_w = warp_scan(w);
          const u64 b = through_parts + __shfl_sync(0xffffffffu, through_w - w, warp) + through - v;
          through_parts += __shfl_sync(0xffffffffu, through_w, 31);
          if (v > 0 && b <= target)
            best = max(best, 1ull << 63 | u64(i));
          else if (const float share = light_share(i, l, lq); share > 0.f)
            best = max(best, u64(__float_as_uint(share)) << 32 | u64(i));
          __syncthreads();
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (lane == 0) sh.warps[warp] = best;
        __syncthreads();
        if (warp == 0) {
          best = sh.warps[lane];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
          if (lane == 0) a.next[r] = int(best & 0xffffffffu);
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
  Args a{logits, draft_logits, token, start, temperature, u, u_sample, M, R, V, accepted, next, static_cast<float2*>(ws), 1, 0, err};
  const int mats = draft_logits ? 2 : 1;
  // Long stretches: a CTA's own 1.5 us are little then; short ones fill the GPU when there are few rows.  Of 8192, 16384,
  // 24576 and 32768 logits: 32 requests of 100003 fp32 logits 20.8, 19.6, 20.8, 22.0 us; 64 of 248320 in bf16 31, 31, 30, 31.
  const int64_t wanted = std::max<int64_t>({V / 16384, 4 * sm_count() / (M * mats), 1});
  a.stretch = int((V + wanted - 1) / std::min<int64_t>(wanted, kMostStretches) + 4095) / 4096 * 4096;
  a.stretches = int((V + a.stretch - 1) / a.stretch);
  const bool pdl = overlap_enabled();
  const bool xb = lt == BL_BF16;
  const dim3 grid(unsigned(M), unsigned(a.stretches), unsigned(mats));
  const cudaError_t e = xb ? launch(verify_mass_kernel<true>, grid, dim3(kMassThreads), 0, s, pdl, a)
                           : launch(verify_mass_kernel<false>, grid, dim3(kMassThreads), 0, s, pdl, a);
  if (e != cudaSuccess) return e;
  // a row in c CTAs: some passes over its share, and the exchanges
  const int c = ctas_per_row(R, [&](int c) { return 8.0 + 1.5 * (c > 1) + double(V) / c * 1e-4; });
  if (xb) return c == 1 ? launch_draw<true, 1>(a, s) : c == 2 ? launch_draw<true, 2>(a, s) : c == 4 ? launch_draw<true, 4>(a, s) : launch_draw<true, 8>(a, s);
  return c == 1 ? launch_draw<false, 1>(a, s) : c == 2 ? launch_draw<false, 2>(a, s) : c == 4 ? launch_draw<false, 4>(a, s) : launch_draw<false, 8>(a, s);
}

}  // namespace bl
