// Residual addition, RMSNorm and absmax int8 quantization of a token, the
// input side of the int8 products:
//   h = rnd(x + residual);  r = fl(1 / sqrt(sum h^2 / K + eps));
//   v = fl(fl(h r) w);  y = rnd(v);  q, s = absmax codes of v (act_quant.cuh).
// The codes have to be the same for every launch shape, so the only quantity
// that depends on an order of additions, the sum of squares, is carried as a
// pair of floats (a two-sum per term: its error is below 2^-40 of the sum)
// and r is rounded to binary32 once; everything after r is elementwise with
// the _rn intrinsics, and a maximum.
//
// Bound: HBM for many tokens (8192 x 5120 bf16 with a residual: 62 us, 69 % of
// the copy rate; the row's two reductions stand between its loads and its
// stores, and 55 registers a thread leave half of the warps), latency for few:
// one token of 2560 2.9 us, of which the launch is most.
#include <cfloat>

#include "act_quant.cuh"
#include "bl_internal.h"

namespace bl {
namespace {

// An unevaluated sum hi + lo.
struct Pair {
  float hi, lo;
};

// p + v, v added without rounding (two-sum); the rounding errors collect in lo.
__device__ __forceinline__ void pair_add(Pair& p, float v) {
  const float t = __fadd_rn(p.hi, v);
  const float z = __fsub_rn(t, p.hi);
  p.lo = __fadd_rn(p.lo, __fadd_rn(__fsub_rn(p.hi, __fsub_rn(t, z)), __fsub_rn(v, z)));
  p.hi = t;
}

__device__ __forceinline__ void pair_add(Pair& p, const Pair& q) {
  pair_add(p, q.hi);
  p.lo = __fadd_rn(p.lo, q.lo);
}

// p + h^2; the square of a bf16 value is exact, that of a float is a pair.
template <bool XB>
__device__ __forceinline__ void pair_add_square(Pair& p, float h) {
  const float sq = __fmul_rn(h, h);
  if (!XB) p.lo = __fadd_rn(p.lo, __fmaf_rn(h, h, -sq));
  pair_add(p, sq);
}

// Sum over groups of `lanes` lanes (a power of two).  A two-sum's error term
// is exact, so the lanes of a pair compute the same result in either order.
__device__ __forceinline__ Pair warp_pair_sum(Pair p, int lanes = 32) {
  for (int o = lanes / 2; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, p.hi, o), lo = __shfl_xor_sync(0xffffffffu, p.lo, o);
    p.lo = __fadd_rn(p.lo, lo);
    pair_add(p, hi);
  }
  return p;
}
__device__ __forceinline__ float warp_max_of(float v, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// fl(1 / sqrt(sum / K + eps)): the mean in pairs (1/K given as one), one
// Newton step from the hardware's approximation whose residual is formed
// exactly, one final rounding.  0 if the mean plus eps is 0.
__device__ __forceinline__ float inv_rms(Pair sum, Pair inv_k, float eps) {
  Pair m;
  m.hi = __fmul_rn(sum.hi, inv_k.hi);
  m.lo = __fmaf_rn(sum.hi, inv_k.hi, -m.hi) + __fmaf_rn(sum.hi, inv_k.lo, __fmul_rn(sum.lo, inv_k.hi));
  pair_add(m, eps);
  const float a = __fadd_rn(m.hi, m.lo);
  const float b = __fsub_rn(m.lo, __fsub_rn(a, m.hi));
  if (a == 0.f) return 0.f;
  const float r = rsqrtf(a);
  const float r2 = __fmul_rn(r, r);
  const float r2l = __fmaf_rn(r, r, -r2);
  const float d = __fsub_rn(__fsub_rn(__fmaf_rn(-a, r2, 1.f), __fmul_rn(a, r2l)), __fmul_rn(b, r2));  // 1 - (a+b) r^2
  return __fmaf_rn(r, d * __fmaf_rn(0.375f, d, 0.5f), r);
}

struct Args {
  const void *x, *res, *w;
  void *h, *y;
  int8_t* q;
  float* s;
  int64_t M, K;
  Pair inv_k;
  float eps;
};

template <bool XB>
__device__ __forceinline__ float load(const void* x, int64_t i) {
  if (XB) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(x)[i]);
  return reinterpret_cast<const float*>(x)[i];
}
template <bool XB>
__device__ __forceinline__ void store(void* x, int64_t i, float v) {
  if (XB)
    reinterpret_cast<uint16_t*>(x)[i] = f32_to_bf16_bits_rn(v);
  else
    reinterpret_cast<float*>(x)[i] = v;
}

// One CTA per token, any K, any alignment; the row is read three times (its
// second and third reads from L2).
template <bool XB>
__global__ void __launch_bounds__(512) rmsnorm_quant_any_kernel(const Args a) {
  __shared__ Pair red[16];
  __shared__ float redm[16];
  const int64_t base = int64_t(blockIdx.x) * a.K;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  pdl_wait();
  Pair p = {0.f, 0.f};
  for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x) {
    float h = load<XB>(a.x, base + k);
    if (a.res) {
      h = __fadd_rn(h, load<XB>(a.res, base + k));
      if (XB) h = bf16_bits_to_f32(f32_to_bf16_bits_rn(h));
    }
    if (a.h) store<XB>(a.h, base + k, h);
    pair_add_square<XB>(p, h);
  }
  p = warp_pair_sum(p);
  if (lane == 0) red[warp] = p;
  __syncthreads();
  p = Pair{0.f, 0.f};
  for (int i = 0; i < nw; ++i) pair_add(p, red[i]);
  const float r = inv_rms(p, a.inv_k, a.eps);
  const void* hr = a.h ? a.h : a.x;  // this thread wrote the elements of h that it reads
  float m = 0.f;
  for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x)
    m = fmaxf(m, fabsf(__fmul_rn(__fmul_rn(load<XB>(hr, base + k), r), load<XB>(a.w, k))));
  m = warp_max(m);
  if (lane == 0) redm[warp] = m;
  __syncthreads();
  m = 0.f;
  for (int i = 0; i < nw; ++i) m = fmaxf(m, redm[i]);
  float sc, inv;
  absmax_scales(m, sc, inv);
  if (threadIdx.x == 0) a.s[blockIdx.x] = sc;
  for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x) {
    const float v = __fmul_rn(__fmul_rn(load<XB>(hr, base + k), r), load<XB>(a.w, k));
    if (a.y) store<XB>(a.y, base + k, v);
    a.q[base + k] = int8_t(quant_code(v, inv));
  }
  pdl_launch_dependents();
}

// Eight elements rounded to bf16 (or as they are) and stored at chunk i of a row.
template <bool XB>
__device__ __forceinline__ void store8(void* row, int i, const float (&v)[8]) {
  if (XB) {
    reinterpret_cast<uint4*>(row)[i] =
        make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
  } else {
    reinterpret_cast<float4*>(row)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(row)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// v rounded to bf16 and widened again, two at a time.
__device__ __forceinline__ void round8(float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint32_t w = bf16x2_rn(v[j], v[j + 1]);
    v[j] = __uint_as_float(w << 16);
    v[j + 1] = __uint_as_float(w & 0xffff0000u);
  }
}

// quant8's codes without its slow conversions: adding 1.5 * 2^23 rounds a
// value of |v inv| < 2^22 to the nearest integer, ties to even, and leaves it
// in the low bits.  |v inv| <= 127 (1 + 2^-22) for a finite inv, so no clamp is
// needed; 127 / max|v| overflows below 3.7e-37.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.f));
  return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

// The row stays in registers: thread t of a token's threads has chunks t, t +
// threads, ... of 8 elements, at most CH of them; everything is read and
// written once.  WARP: a warp per token, eight tokens per CTA (no barriers);
// otherwise a CTA per token, whose sums and maxima meet in shared memory.
// 16-byte aligned rows, K % 8 == 0.
//
// The thread's sum starts from its largest square m0, which is taken off
// again: then no term exceeds the sum so far, and the rounding error of an
// addition is (v - (t - hi)), four operations instead of seven.
//
// Bound: HBM, with the arithmetic close behind: about 20 operations per
// element of the 23 that the SMs issue in the time its 7 bytes take.
template <bool XB, int CH, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rmsnorm_quant_rows_kernel(const Args a) {
  __shared__ Pair red[WARP ? 1 : 32];
  __shared__ float redm[WARP ? 1 : 32];
  constexpr int kBytes = XB ? 2 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m = WARP ? int64_t(blockIdx.x) * 8 + warp : blockIdx.x;
  const int t = WARP ? lane : threadIdx.x, threads = WARP ? 32 : blockDim.x, nw = blockDim.x >> 5;
  const int n8 = int(a.K / 8);
  if (WARP && m >= a.M) return;  // whole warps; no barrier follows
  pdl_wait();
  const int64_t at = m * a.K * kBytes;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + at;
  const uint8_t* res = a.res ? static_cast<const uint8_t*>(a.res) + at : nullptr;
  uint8_t* h = a.h ? static_cast<uint8_t*>(a.h) + at : nullptr;
  uint8_t* y = a.y ? static_cast<uint8_t*>(a.y) + at : nullptr;
  float v[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = t + c * threads;
    if (i < n8) load8<XB>(x, i, v[c]);
  }
  if (res) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = t + c * threads;
      if (i < n8) {
        float r[8];
        load8<XB>(res, i, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = __fadd_rn(v[c][j], r[j]);
        if (XB) round8(v[c]);
      }
    }
  }
  float m0 = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = t + c * threads;
    if (i < n8) {
      if (h) store8<XB>(h, i, v[c]);
#pragma unroll
      for (int j = 0; j < 8; ++j) m0 = fmaxf(m0, fabsf(v[c][j]));
    }
  }
  m0 = __fmul_rn(m0, m0);
  Pair p = {m0, 0.f};
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (t + c * threads < n8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float sq = __fmul_rn(v[c][j], v[c][j]);
        if (!XB) p.lo = __fadd_rn(p.lo, __fmaf_rn(v[c][j], v[c][j], -sq));
        const float sum = __fadd_rn(p.hi, sq);
        p.lo = __fadd_rn(p.lo, __fsub_rn(sq, __fsub_rn(sum, p.hi)));
        p.hi = sum;
      }
    }
  pair_add(p, -m0);
  p = warp_pair_sum(p);
  int lanes = 1;  // that hold the warps' sums, several times over
  if (!WARP) {
    while (lanes < nw) lanes *= 2;
    if (lane == 0) red[warp] = p;
    __syncthreads();
    const int w = lane & (lanes - 1);
    p = warp_pair_sum(w < nw ? red[w] : Pair{0.f, 0.f}, lanes);
  }
  const float r = inv_rms(p, a.inv_k, a.eps);
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = t + c * threads;
    if (i < n8) {
      float w[8];
      load8<XB>(a.w, i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[c][j] = __fmul_rn(__fmul_rn(v[c][j], r), w[j]);
        most = fmaxf(most, fabsf(v[c][j]));
      }
      if (y) store8<XB>(y, i, v[c]);
    }
  }
  most = warp_max(most);
  if (!WARP) {
    if (lane == 0) redm[warp] = most;
    __syncthreads();
    const int w = lane & (lanes - 1);
    most = warp_max_of(w < nw ? redm[w] : 0.f, lanes);
  }
  float inv = most == 0.f ? 0.f : __fdiv_rn(127.f, most);  // absmax_scales, its scale by one thread
  if (inv > FLT_MAX) {  // codes8 has no clamp
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = float(quant_code(v[c][j], inv));
    inv = 1.f;
  }
  if (t == 0) {
    float sc, unused;
    absmax_scales(most, sc, unused);
    a.s[m] = sc;
  }
  uint2* q = reinterpret_cast<uint2*>(a.q + m * a.K);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = t + c * threads;
    if (i < n8) q[i] = codes8(v[c], inv);
  }
  pdl_launch_dependents();
}

template <bool XB, int CH>
cudaError_t launch_rows(const Args& a, cudaStream_t s, bool pdl) {
  const int64_t n8 = a.K / 8;
  if (n8 <= 32 * CH && CH <= 4)
    return launch(rmsnorm_quant_rows_kernel<XB, CH, true>, dim3(unsigned((a.M + 7) / 8)), dim3(256), 0, s, pdl, a);
  const unsigned threads = unsigned(((n8 + CH - 1) / CH + 31) / 32 * 32);
  return launch(rmsnorm_quant_rows_kernel<XB, CH, false>, dim3(unsigned(a.M)), dim3(threads), 0, s, pdl, a);
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const void* x, const void* residual, bl_dtype xt, const void* rms_w, float eps,
                                 int64_t M, int64_t K, void* h, void* y, int8_t* q, float* sc, cudaStream_t s) {
  Args a{x, residual, rms_w, h, y, q, sc, M, K, {}, eps};
  a.inv_k.hi = float(1.0 / double(K));
  a.inv_k.lo = float(1.0 / double(K) - double(a.inv_k.hi));
  const bool pdl = overlap_enabled();
  const bool xb = xt == BL_BF16;
  const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                        reinterpret_cast<uintptr_t>(rms_w) | reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(y);
  if (K % 8 == 0 && (all & 15) == 0 && (reinterpret_cast<uintptr_t>(q) & 7) == 0 && K <= 32768) {
    // Chunks per thread: for few tokens one while a row then has at most 512 threads (the shortest chain),
    // for many four: a warp's share of the two reductions costs as much as 8 elements per lane (8192 x 5120
    // bf16: 320 threads with two chunks 67 us, 160 with four 62 us).
    const int64_t n8 = K / 8;
    const bool many = M > 2 * sm_count();
    if (n8 <= 512 && !many) return xb ? launch_rows<true, 1>(a, s, pdl) : launch_rows<false, 1>(a, s, pdl);
    if (n8 <= 1024 && !many) return xb ? launch_rows<true, 2>(a, s, pdl) : launch_rows<false, 2>(a, s, pdl);
    return xb ? launch_rows<true, 4>(a, s, pdl) : launch_rows<false, 4>(a, s, pdl);
  }
  if (xb) return launch(rmsnorm_quant_any_kernel<true>, dim3(unsigned(M)), dim3(512), 0, s, pdl, a);
  return launch(rmsnorm_quant_any_kernel<false>, dim3(unsigned(M)), dim3(512), 0, s, pdl, a);
}

}  // namespace bl
