// Rotary positions and the cache's new rows (bl_rope_append): of a token's row
// (q heads, k heads, v heads) the q and k heads are turned by the token's angle,
//   a' = a cos - b sin,  b' = b cos + a sin
// for coordinates i and i + rotary / 2, in fp32 and rounded to bf16 once; q goes to
// q, k and v to row `slot` of the paged cache.
//
// An item is VEC pairs of a head, or VEC coordinates that are only copied; a CTA
// takes the items of a few tokens.
//
// Bound: HBM for prompts, launch and two dependent reads (position, angle) for few tokens.
#include "bl_device.cuh"
#include "bl_internal.h"

namespace bl {
namespace {

constexpr int kThreads = 256;

struct Args {
  const void* x;
  const float *cos, *sin;
  const int32_t *position, *slot;
  uint16_t *q, *k, *v;
  int64_t M, positions, slots;
  int H, Hk, D, half, page, tokens;  // tokens: per CTA
  unsigned int* err;
};

template <bool XB, int VEC>
__device__ __forceinline__ void load(const void* x, int64_t i, float (&v)[VEC]) {
  if (VEC == 1) {
    v[0] = XB ? bf16_bits_to_f32(static_cast<const uint16_t*>(x)[i]) : static_cast<const float*>(x)[i];
  } else if (XB) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const float4 f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i)[j];
      v[4 * j] = f.x, v[4 * j + 1] = f.y, v[4 * j + 2] = f.z, v[4 * j + 3] = f.w;
    }
  }
}

template <int VEC>
__device__ __forceinline__ void store(uint16_t* y, int64_t i, const float (&v)[VEC]) {
  if (VEC == 1) {
    y[i] = f32_to_bf16_bits_rn(v[0]);
  } else {
    uint32_t u[VEC / 2 > 0 ? VEC / 2 : 1];
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) u[j] = bf16x2_rn(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<uint4*>(y + i) = make_uint4(u[0], u[VEC > 2 ? 1 : 0], u[VEC > 4 ? 2 : 0], u[VEC > 6 ? 3 : 0]);
  }
}

template <bool XB, int VEC>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const Args a) {
  const int pairs = a.half / VEC, rest = (a.D - 2 * a.half) / VEC;  // items of a turned head
  const int turned = (a.H + a.Hk) * (pairs + rest), copied = a.Hk * (a.D / VEC);
  const int items = turned + copied, heads = a.H + 2 * a.Hk;
  const int64_t first = int64_t(blockIdx.x) * a.tokens;
  const int mine = int(min(int64_t(a.tokens), a.M - first));
  bool bad = false;
  pdl_wait();
  for (int at = threadIdx.x; at < mine * items; at += kThreads) {
    const int64_t m = first + at / items;
    const int item = at % items;
    const int position = a.position[m], slot = a.slot[m];
    if (position < 0) continue;  // no token
    if (position >= a.positions || slot >= a.slots) bad = true;
    if (position >= a.positions) continue;
    int head, i;  // head of the row, coordinate in it
    bool pair = false;
    if (item < turned) {
      const int j = item % (pairs + rest);
      head = item / (pairs + rest);
      pair = j < pairs;
      i = pair ? j * VEC : 2 * a.half + (j - pairs) * VEC;
    } else {
      head = a.H + a.Hk + (item - turned) / (a.D / VEC);
      i = (item - turned) % (a.D / VEC) * VEC;
    }
    uint16_t* to = nullptr;
    if (head < a.H) {
      to = a.q + (m * a.H + head) * a.D;
    } else if (slot >= 0 && slot < a.slots) {
      const int h = head - a.H < a.Hk ? head - a.H : head - a.H - a.Hk;
      to = (head - a.H < a.Hk ? a.k : a.v) + ((int64_t(slot / a.page) * a.Hk + h) * a.page + slot % a.page) * a.D;
    }
    if (!to) continue;
    const int64_t from = (m * heads + head) * a.D + i;
    float v[VEC];
    load<XB, VEC>(a.x, from, v);
    if (pair) {
      float w[VEC], c[VEC], s[VEC];
      load<XB, VEC>(a.x, from + a.half, w);
      load<false, VEC>(a.cos, int64_t(position) * a.half + i, c);
      load<false, VEC>(a.sin, int64_t(position) * a.half + i, s);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float t = __fmaf_rn(v[j], c[j], -__fmul_rn(w[j], s[j]));
        w[j] = __fmaf_rn(w[j], c[j], __fmul_rn(v[j], s[j]));
        v[j] = t;
      }
      store<VEC>(to, i + a.half, w);
    }
    store<VEC>(to, i, v);
  }
  if (bad) atomicOr(a.err, BL_DEVERR_RANGE);
  pdl_launch_dependents();
}

template <bool XB, int VEC>
cudaError_t launch_as(const Args& a, cudaStream_t s) {
  const int64_t grid = (a.M + a.tokens - 1) / a.tokens;
  return launch(rope_append_kernel<XB, VEC>, dim3(unsigned(grid)), dim3(kThreads), 0, s, overlap_enabled(), a);
}

}  // namespace

cudaError_t launch_rope_append(const void* qkv, bl_dtype xt, const float* cos, const float* sin, const int32_t* position,
                               const int32_t* slot, int64_t M, int H, int Hk, int D, int rotary, int64_t positions,
                               uint16_t* q, uint16_t* k_cache, uint16_t* v_cache, int64_t pages, int page, cudaStream_t s) {
  unsigned int* err = dev_error_ptr();
  if (!err) return cudaErrorUnknown;
  Args a{qkv, cos, sin, position, slot, q, k_cache, v_cache, M, positions, pages * page, H, Hk, D, rotary / 2, page, 1, err};
  a.tokens = M > 8 * sm_count() ? 4 : 1;
  const bool wide = a.half % 8 == 0 && ((reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) & 15) == 0;
  if (xt == BL_BF16) return wide ? launch_as<true, 8>(a, s) : launch_as<true, 1>(a, s);
  return wide ? launch_as<false, 8>(a, s) : launch_as<false, 1>(a, s);
}

}  // namespace bl
