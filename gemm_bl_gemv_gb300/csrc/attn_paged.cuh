// Shared by the kernels of bl_attn_paged: units, tiles, the places of both, and the joining of parts.
#pragma once
#include "bl_device.cuh"
#include "bl_internal.h"
#include "paged.cuh"

namespace bl {
namespace attn {

constexpr int TERMS = 3;        // of a weight: bf16 numbers that it enters the second product in, 24 bits
constexpr int kMostCtas = 160;  // of the first kernel, for the size of the workspace

// Rows of a unit: n from row0 on, of a request's new tokens from `token` on and a key-value head.
struct Unit {
  int token, head, row0, n;
};
// Division of 0 <= n < 2^31 by a number known at launch.
struct Divisor {
  uint32_t mul, shift, d;
  void set(uint32_t by) {  // mul = ceil(2^(31 + shift) / by), 2^(shift - 1) < by <= 2^shift
    d = by;
    for (shift = 0; (uint64_t(1) << shift) < by;) ++shift;
    mul = uint32_t(((uint64_t(1) << (31 + shift)) + by - 1) / by);
  }
  __device__ __forceinline__ int quotient(int n) const { return int(__umulhi(2 * uint32_t(n), mul) >> shift); }
};
// a / b for a >= 0, b > 0: 64-bit divisions take some 400 clocks, and small numbers do not need them.
static __device__ __noinline__ int64_t long_quotient(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if ((a | b) >> 31 == 0) return uint32_t(a) / uint32_t(b);
  return long_quotient(a, b);
}
// What a CTA leaves of the unit that goes on in the next CTA's stretch.
struct __align__(16) Header {
  Unit unit;
  int present;
  int follow;  // CTAs after this one that have a part
  int pad[2];
};
struct Args {
  const uint16_t *q, *k, *v;
  const int32_t *table, *length, *start;
  void* out;
  Header* header;
  float2* stat;  // (max, sum) of each row of each part: two parts of every CTA, then one of every warp
  float* acc;    // weighted sums
  int64_t M, R, pages, W;
  int H, Hk, G, D, page, rows;  // rows: kept of a part
  int64_t window, sinks;
  float scale;    // |scale| log2(e), of the queries times `sign`
  uint32_t sign;  // xor on a pair of queries
  bool zero;      // a scale of 0: so are the queries
  Divisor by_page, by_group;
  bool tiled;  // a tile lies within a page
  unsigned long long wait_ns;  // a test limit of the roles' waits, or 0
  unsigned int* err;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A request: its rows, and which tiles its new tokens see.
struct Request {
  int first, n, length;   // new tokens; tokens in the cache
  int low;                // from here on the first new token's window sees the cache
  int early, low_tile;    // tiles of the first tokens; the window's first tile
  int tiles, blocks;      // of a unit; units per head
  bool bad;
};
template <class S>
__device__ __noinline__ Request request_of(const Args& a, int64_t r) {
  Request q;
  const Rows rows = rows_of(a.start, r, a.M);
  q.first = rows.first;
  q.n = rows.n;
  const int64_t most = min(a.W * a.page, int64_t(INT32_MAX - 255));  // so that a tile's tokens have numbers
  const int given = a.length[r];
  q.length = int(max(int64_t(0), min(int64_t(given), most)));
  q.bad = rows.bad || q.length != given;
  q.low = a.window > 0 ? int(max(int64_t(0), int64_t(q.length) - q.n + 1 - a.window)) : 0;
  q.low_tile = q.low / S::TT;
  q.early = int(min(int64_t(q.low_tile), (min(a.sinks, int64_t(q.low)) + S::TT - 1) / S::TT));
  const int64_t end = (int64_t(q.length) + S::TT - 1) / S::TT;
  q.tiles = max(1, int(q.early + end - q.low_tile));
  q.blocks = int((int64_t(q.n) * a.G + S::ROWS - 1) / S::ROWS);
  return q;
}

// Where a row of a unit lies in q and out.
__device__ __forceinline__ int64_t row_at(const Args& a, const Unit& u, int row) {
  const int t = a.by_group.quotient(u.row0 + row), h = u.row0 + row - t * a.G;
  return ((int64_t(u.token) + t) * a.H + u.head * a.G + h) * a.D;
}

// Joins a row's parts by a warp: stat(p) and acc(p) of parts 0..n-1; out(l, top, o) gets the result, lane by lane four
// columns from 4 lane + 128 i on.
template <class Stat, class Acc, class Out>
__device__ __forceinline__ void join_row(const Args& a, int n, Stat stat, Acc acc, Out out) {
  const int lane = threadIdx.x & 31;
  float2 s = lane < n ? stat(lane) : make_float2(-INFINITY, 0.f);
  float top = s.x;
  for (int p = lane + 32; p < n; p += 32) top = fmaxf(top, stat(p).x);
  top = warp_max(top);
  const float base = top == -INFINITY ? 0.f : top;
  float l = 0.f;
  float4 o[2] = {};
  for (int p0 = 0; p0 < n; p0 += 32) {
    float f = 0.f;
    if (p0 + lane < n) {
      if (p0 > 0) s = stat(p0 + lane);
      f = exp2_fast((s.x - base) * a.scale);
      l = __fmaf_rn(f, s.y, l);
    }
    const int m = min(32, n - p0);
#pragma unroll 1
    for (int p = 0; p < m; p += 8) {  // eight loads at a time
      float4 y[8][2];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          y[j][i] = p + j < m && lane + 32 * i < a.D / 4 ? reinterpret_cast<const float4*>(acc(p0 + p + j))[lane + 32 * i]
                                                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float fp = __shfl_sync(0xffffffffu, f, (p + j) & 31);
        if (p + j < m) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            o[i].x = __fmaf_rn(fp, y[j][i].x, o[i].x);
            o[i].y = __fmaf_rn(fp, y[j][i].y, o[i].y);
            o[i].z = __fmaf_rn(fp, y[j][i].z, o[i].z);
            o[i].w = __fmaf_rn(fp, y[j][i].w, o[i].w);
          }
        }
      }
    }
  }
  l = warp_sum(l);
  out(l, top, o);
}

// The row's result, of a joined row.
template <bool F32>
__device__ __forceinline__ void store_row(const Args& a, int64_t to, float l, float top, const float4 (&o)[2]) {
  const int lane = threadIdx.x & 31;
  const float inv = top == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < a.D / 4) {
      const int64_t d = to + (lane + 32 * i) * 4;
      if (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + d) = make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + d) =
            make_uint2(bf16x2_rn(o[i].x * inv, o[i].y * inv), bf16x2_rn(o[i].z * inv, o[i].w * inv));
    }
}

// A place in the sequence of all tiles.
template <class S>
struct Place {
  int64_t r;
  Request q;
  int unit, tile;  // of the request; of the unit

  __device__ __forceinline__ int head() const { return q.blocks == 1 ? unit : unit / q.blocks; }
  __device__ __forceinline__ int row0() const { return q.blocks == 1 ? 0 : unit % q.blocks * S::ROWS; }
  __device__ __forceinline__ int token() const {
    return (tile < q.early ? tile : q.low_tile + tile - q.early) * S::TT;
  }
  // The tile t0 < before[n]; before[i]: tiles before request i * share.
  __device__ __forceinline__ void find(const Args& a, const int64_t* before, int n, int64_t share, int64_t t0) {
    int lo = 0, hi = n;  // before[lo] <= t0 < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= t0)
        lo = mid;
      else
        hi = mid;
    }
    int64_t rest = t0 - before[lo];
    for (r = lo * share;; ++r) {
      q = request_of<S>(a, r);
      const int64_t all = int64_t(a.Hk) * q.blocks * q.tiles;
      if (rest < all) break;
      rest -= all;
    }
    unit = int(quotient(rest, q.tiles));
    tile = int(rest - int64_t(unit) * q.tiles);
  }
  // To the next tile; there must be one.
  __device__ __forceinline__ void next(const Args& a) {
    if (++tile < q.tiles) return;
    tile = 0;
    if (++unit < a.Hk * q.blocks) return;
    unit = 0;
    do {
      q = request_of<S>(a, ++r);
    } while (q.blocks == 0 && r + 1 < a.R);
  }
};

// The kernel of attn_paged_tc.cu: D <= 128, 32 rows to a unit; cudaErrorNotSupported, having launched nothing, for pages
// that it has no boxes for.
cudaError_t launch_tc(const Args& a, int grid, bool f32, cudaStream_t s);

}  // namespace attn
}  // namespace bl
