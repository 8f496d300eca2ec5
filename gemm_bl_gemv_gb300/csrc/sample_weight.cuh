// Order and weight of a logit, shared by the sampling kernels.
//   key(l)    : unsigned, rising with l (NaN as -inf, -0 as 0).
//   weight(l) : exp((l - max) / T) as an integer in units of 2^-44.
#pragma once
#include "bl_device.cuh"

namespace bl {

constexpr int kWeightBits = 44;  // the largest weight is 2^44, so 2^19 of them stay below 2^64
constexpr float kGreedyBelow = 1e-5f;

__device__ __forceinline__ uint32_t key_of_f32(float l) {
  const uint32_t b = __float_as_uint(l != l ? -INFINITY : l + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float f32_of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// log2(e) / T as a pair of floats; greedy: hi < 0.
struct Slope {
  float hi, lo;
};
__device__ __forceinline__ Slope slope_of(float t) {
  if (!(t >= kGreedyBelow)) return Slope{-1.f, 0.f};
  const float lh = 1.44269502162933349609375f;         // log2(e) to 24 bits
  const float ll = 1.92596303313e-8f;                  // log2(e) - lh
  const float q = __fdiv_rn(lh, t);
  const float rest = __fadd_rn(__fmaf_rn(-q, t, lh), ll);  // lh - q t is exact
  return Slope{q, q > 0.f ? __fdiv_rn(rest, t) : 0.f};
}

// 2^(j/32) in units of 2^-44, j = -16..16, rounded to nearest.
constexpr int kExp2Entries = 33;
__constant__ unsigned long long kExp2[kExp2Entries] = {
    12439554047902ull, 12711944812080ull, 12990300157313ull, 13274750690919ull, 13565429880144ull,
    13862474114787ull, 14166022771192ull, 14476218277651ull, 14793206181226ull, 15117135216047ull,
    15448157373097ull, 15786427971528ull, 16132105731538ull, 16485352848846ull, 16846335070792ull,
    17215221774115ull, 17592186044416ull, 17977404757381ull, 18371058661769ull, 18773332464219ull,
    19184414915921ull, 19604498901178ull, 20033781527906ull, 20472464220127ull, 20920752812471ull,
    21378857646762ull, 21846993670708ull, 22325380538761ull, 22814242715178ull, 23313809579344ull,
    23824315533396ull, 24346000112214ull, 24879108095804ull};

// The table in shared memory (lanes read different entries), with each entry
// in units of 2^8 as a float.
struct Exp2Table {
  ulonglong2 v[kExp2Entries];
};

// By the whole CTA; the caller synchronizes.
__device__ __forceinline__ void fill_exp2_table(Exp2Table& t) {
  for (int j = threadIdx.x; j < kExp2Entries; j += blockDim.x)
    t.v[j] = make_ulonglong2(kExp2[j], __float_as_uint(__ull2float_rn(kExp2[j] >> 8)));
}

// 2^(e + el) in units of 2^-44, e <= 0 and |el| small, e and el a pair: 2^n 2^(j/32)
// 2^r, |r| <= 1/64: the power of two is a shift, 2^(j/32) comes from the table, and
// 2^r - 1 <= 2^-6.5 is a polynomial in float, whose 2^-24 relative error leaves about
// 2^-30 of the weight.  0 for e <= -63, NaN, or where `none` is given.
// `shift` receives -n: the result is not shifted yet.  No branches: callers
// have several in flight.
__device__ __forceinline__ unsigned long long exp2_mantissa(float e, float el, bool none, const Exp2Table& t, int& shift) {
  none |= !(e > -63.f);
  e = none ? 0.f : e;
  const float n = rintf(e);                 // -63..0
  const float f = __fsub_rn(e, n);          // exact, |f| <= 1/2
  const float j = rintf(f * 32.f);          // -16..16
  const float r = __fmaf_rn(j, -0.03125f, f) + el;
  // 2^r - 1 = a + a^2 / 2 + a^3 / 6 + a^4 / 24 with a = r ln 2
  const float a = r * 0.693147180559945f;
  const float p = a * __fmaf_rn(a, __fmaf_rn(a, __fmaf_rn(a, 0.041666667f, 0.16666667f), 0.5f), 1.f);
  const ulonglong2 base = t.v[int(j) + 16];
  // base < 2^45, so |p base| < 2^39: in units of 2^8 it is a signed 32-bit integer
  const long long more = static_cast<long long>(__float2int_rn(p * __uint_as_float(uint32_t(base.y)))) * 256;
  shift = -int(n);                          // 0..63
  return none ? 0ull : base.x + static_cast<unsigned long long>(more);
}

// (l - max) log2(e) / T as a pair of floats.
struct Pair {
  float e, el;
};
__device__ __forceinline__ Pair exponent_of(float l, float top, Slope c) {
  const float d = __fsub_rn(l, top);  // < 0; its rounding error is dl
  const float z = __fsub_rn(d, l);
  const float dl = __fadd_rn(__fsub_rn(l, __fsub_rn(d, z)), __fsub_rn(-top, z));
  const float e = __fmul_rn(d, c.hi);
  return {e, __fmaf_rn(d, c.hi, -e) + __fmaf_rn(d, c.lo, __fmul_rn(dl, c.hi))};
}

// The weight of logit l.
__device__ __forceinline__ unsigned long long weight_mantissa(float l, float top, Slope c, const Exp2Table& t,
                                                              int& shift) {
  const Pair x = exponent_of(l, top, c);
  // no weight: too small, greedy, -inf, NaN, beside +inf
  const unsigned long long w = exp2_mantissa(x.e, x.el, c.hi < 0.f, t, shift);
  shift = l == top ? 0 : shift;
  return l == top ? 1ull << kWeightBits : w;
}

__device__ __forceinline__ unsigned long long weight_of(float l, float top, Slope c, const Exp2Table& t) {
  int shift;
  const unsigned long long w = weight_mantissa(l, top, c, t, shift);
  return (w + ((1ull << shift) >> 1)) >> shift;
}

// The share of logit l's weight in `kept`; the weight keeps its full precision here.
__device__ __forceinline__ float share_of(float l, float top, Slope c, const Exp2Table& t, unsigned long long kept) {
  int shift;
  const unsigned long long w = weight_mantissa(l, top, c, t, shift);
  return float(double(w) * double(exp2i(-shift)) / double(kept));
}

// p * mass for 0 <= p < 1, rounded down (rest: whether a fraction was dropped),
// in integers: exact, and no use of the slow fp64 pipe by a whole CTA.
__device__ __forceinline__ unsigned long long scaled(float p, unsigned long long mass, bool& rest) {
  const uint32_t b = __float_as_uint(p);
  const uint32_t e = b >> 23;
  const unsigned long long mant = (b & 0x7fffffu) | (e ? 0x800000u : 0u);  // p = mant 2^-sh, sh >= 24
  const int sh = 150 - int(e ? e : 1u);
  const unsigned long long lo = mass * mant, hi = __umul64hi(mass, mant);
  if (sh < 64) {
    rest = (lo << (64 - sh)) != 0;
    return hi << (64 - sh) | lo >> sh;
  }
  if (sh < 128) {
    rest = lo != 0 || (hi & ((1ull << (sh - 64)) - 1)) != 0;
    return hi >> (sh - 64);
  }
  rest = (lo | hi) != 0;
  return 0;
}

// ceil(p * mass) for 0 <= p < 1, and floor(u * mass) for 0 <= u < 1, mass > 0.
__device__ __forceinline__ unsigned long long mass_limit(float p, unsigned long long mass) {
  bool rest;
  const unsigned long long q = scaled(p, mass, rest);
  return q + rest;
}
__device__ __forceinline__ unsigned long long mass_target(float u, unsigned long long mass) {
  bool rest;
  return scaled(u, mass, rest);
}

// A row's parameters as given (loaded early, used late).
struct RowValues {
  float temperature, top_p, min_p, u;
  int top_k;
  __device__ __forceinline__ RowValues(int64_t m, const float* t, const int32_t* k, const float* p, const float* mp,
                                       const float* uniform)
      : temperature(t ? t[m] : 1.f), top_p(p ? p[m] : 1.f), min_p(mp ? mp[m] : 0.f), u(uniform[m]), top_k(k ? k[m] : 0) {}
};

// They after clamping.
struct RowFilter {
  Slope slope;
  long long top_k;           // tokens that stay by count
  float top_p, u;            // top_p = 2: no limit
  unsigned long long min_w;  // smallest weight that stays (0: no limit)
};

__device__ __forceinline__ RowFilter row_filter(const RowValues& r, int64_t V) {
  constexpr unsigned long long kOne = 1ull << kWeightBits;
  RowFilter f;
  f.slope = slope_of(r.temperature);
  f.top_k = (r.top_k <= 0 || r.top_k > V) ? V : r.top_k;
  if (r.min_p > 1.f) f.top_k = 1;  // no weight reaches it, so the first token alone stays, whatever ties with it
  f.top_p = r.top_p < 1.f ? fmaxf(r.top_p, 0.f) : 2.f;
  f.min_w = r.min_p > 0.f ? (r.min_p < 1.f ? mass_limit(r.min_p, kOne) : kOne) : 0ull;
  f.u = r.u > 0.f ? fminf(r.u, 0.99999994f) : 0.f;
  return f;
}

}  // namespace bl
