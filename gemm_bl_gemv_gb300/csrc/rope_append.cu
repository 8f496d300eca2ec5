// Rotary positions and the cache's new rows (bl_rope_append): of a token's row
// (q heads, k heads, v heads) the q and k heads are turned by the token's angle,
//   a' = a cos - b sin,  b' = b cos + a sin
// for coordinates i and i + rotary / 2, in fp32 and rounded to bf16 once; q goes to
// q, k and v to row `slot` of the paged cache.
//
// Bound: HBM for prompts, launch and two dependent reads (position, angle) for few tokens: one token 2.2 us, 311 of 56
// heads in fp32 3.6 us, 8192 of 30 heads in bf16 27 us (4.8 TB/s; a copy of the same bytes takes 21.5 us).  Where the rotary
// part or the tables allow no vector loads, one value at a time: 8.7, 16 and 149 us.
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
  int H, Hk, D, half, page;
  unsigned int* err;
};

// VEC values as they lie in memory.
template <bool XB, int VEC>
struct Raw {
  static constexpr int W = VEC == 1 ? 1 : VEC * (XB ? 2 : 4) / 4;
  uint32_t u[W];
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    if (VEC == 1) {
      u[0] = XB ? uint32_t(static_cast<const uint16_t*>(x)[i]) << 16 : static_cast<const uint32_t*>(x)[i];
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + i * (XB ? 2 : 4));
#pragma unroll
      for (int j = 0; j < W / 4; ++j) {
        const uint4 v = p[j];
        u[4 * j] = v.x, u[4 * j + 1] = v.y, u[4 * j + 2] = v.z, u[4 * j + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    return __uint_as_float(VEC == 1 || !XB ? u[j] : j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
  }
};

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

// A token's threads: blockDim.x; thread t turns chunk t % pairs of every few heads, so it reads its angles once.  The
// first loads of a row go out before its position and slot are there.
template <bool XB, int VEC>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const Args a) {
  const int64_t m = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  const int t = threadIdx.x, threads = blockDim.x;
  const int pairs = a.half / VEC, heads = a.H + 2 * a.Hk, turned = a.H + a.Hk;
  const int groups = max(1, threads / pairs);              // heads that are turned at a time
  const int group = pairs < threads ? t / pairs : 0;
  const int rest = (a.D - 2 * a.half) / VEC, all = a.D / VEC;
  const int first = turned * rest, items = first + a.Hk * all;  // what is only copied: the turned heads' rest, then v
  const int64_t from = m * heads * a.D;
  bool bad = false;
  pdl_wait();
  if (m < a.M) {
    const int position = a.position[m], slot = a.slot[m];
    Raw<XB, VEC> v, w, c;
    auto load_pair = [&](int head, int chunk) {
      if (head < turned && group < groups) {
        const int64_t i = from + int64_t(head) * a.D + chunk * VEC;
        v.load(a.x, i);
        w.load(a.x, i + a.half);
      }
    };
    auto item = [&](int at, int& head, int& i) {
      head = at < first ? at / rest : turned + (at - first) / all;
      i = at < first ? 2 * a.half + at % rest * VEC : (at - first) % all * VEC;
    };
    auto load_item = [&](int at) {
      if (at >= items) return;
      int head, i;
      item(at, head, i);
      c.load(a.x, from + int64_t(head) * a.D + i);
    };
    const int chunk0 = t % min(pairs, threads);
    load_pair(group, chunk0);
    load_item(t);
    const bool stored = slot >= 0 && slot < a.slots;
    bad = position >= a.positions || (position >= 0 && slot >= a.slots);
    if (position >= 0 && position < a.positions) {
      const int64_t row = stored ? (int64_t(slot / a.page) * a.Hk * a.page + slot % a.page) * a.D : 0;
      const int64_t head_rows = int64_t(a.page) * a.D;
      // where a head's result goes; nullptr: nowhere
      auto place = [&](int head) -> uint16_t* {
        if (head < a.H) return a.q + (m * a.H + head) * a.D;
        if (!stored) return nullptr;
        return head < turned ? a.k + row + (head - a.H) * head_rows : a.v + row + (head - turned) * head_rows;
      };
      for (int chunk = chunk0; chunk < pairs && group < groups; chunk += threads) {  // one chunk, unless a head has more than the threads
        Raw<false, VEC> cs, sn;
        cs.load(a.cos, int64_t(position) * a.half + chunk * VEC);
        sn.load(a.sin, int64_t(position) * a.half + chunk * VEC);
        for (int head = group; head < turned; head += groups) {
          if (head != group || chunk != chunk0) load_pair(head, chunk);
          uint16_t* to = place(head);
          if (!to) continue;
          float x[VEC], y[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float p = v.get(j), q = w.get(j), co = cs.get(j), si = sn.get(j);
            x[j] = __fmaf_rn(p, co, -__fmul_rn(q, si));
            y[j] = __fmaf_rn(q, co, __fmul_rn(p, si));
          }
          store<VEC>(to, chunk * VEC, x);
          store<VEC>(to, chunk * VEC + a.half, y);
        }
      }
      for (int at = t; at < items; at += threads) {
        if (at != t) load_item(at);
        int head, i;
        item(at, head, i);
        uint16_t* to = place(head);
        if (!to) continue;
        float x[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = c.get(j);
        store<VEC>(to, i, x);
      }
    }
  }
  if (bad && t == 0) atomicOr(a.err, BL_DEVERR_RANGE);
  pdl_launch_dependents();
}

template <bool XB, int VEC>
cudaError_t launch_as(const Args& a, cudaStream_t s) {
  // Few tokens: as many threads as a CTA has for each, so that a thread makes one trip; many: 64, whose angles serve several
  // heads, in small CTAs, whose last ones end together.  256 / 64 threads in us, 56 heads: bf16 400 tokens 3.4 / 4.8, 1200
  // 8.7 / 8.7, 2000 14.4 / 12.8, 4000 25.8 / 22.5; fp32 1200 11.0 / 11.8, 2000 16.7 / 16.1, 4000 30.2 / 29.1.
  const bool many = a.M > 8 * sm_count();
  const unsigned per = many ? 64 : kThreads, tokens = many ? 2 : 1;
  return launch(rope_append_kernel<XB, VEC>, dim3(unsigned((a.M + tokens - 1) / tokens)), dim3(per, tokens), 0, s, overlap_enabled(), a);
}

}  // namespace

cudaError_t launch_rope_append(const void* qkv, bl_dtype xt, const float* cos, const float* sin, const int32_t* position,
                               const int32_t* slot, int64_t M, int H, int Hk, int D, int rotary, int64_t positions,
                               uint16_t* q, uint16_t* k_cache, uint16_t* v_cache, int64_t pages, int page, cudaStream_t s) {
  unsigned int* err = dev_error_ptr();
  if (!err) return cudaErrorUnknown;
  const Args a{qkv, cos, sin, position, slot, q, k_cache, v_cache, M, positions, pages * page, H, Hk, D, rotary / 2, page, err};
  const bool wide = a.half % 8 == 0 && ((reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) & 15) == 0;
  if (xt == BL_BF16) return wide ? launch_as<true, 8>(a, s) : launch_as<true, 1>(a, s);
  return wide ? launch_as<false, 8>(a, s) : launch_as<false, 1>(a, s);
}

}  // namespace bl
