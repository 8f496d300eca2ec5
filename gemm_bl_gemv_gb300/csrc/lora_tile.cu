// Low-rank adapters of long runs of tokens (bl_lora_add), on the 5th-generation
// tensor cores (tcgen05), bf16 activations:
//   y[m,n] = base[m,n] + scale[a] * sum_r B[a,n,r] (sum_k A[a,r,k] x[m,k]).
//
// A cluster of CL CTAs takes 128 tokens.  A run is a stretch of those tokens
// with one adapter; a tile of more than kTileRuns runs is left to the kernel
// for scattered tokens.
//   1. Down: each CTA takes a part of K.  x (128 x 64 blocks) and the run's A
//      (rank x 64) come by TMA through a ring; the tensor core forms the
//      128 x rank product in TMEM, and the rows of the run go to shared
//      memory as fp32.  The CTAs add their parts up in rank order through
//      distributed shared memory, so the sum over K is never rounded below
//      fp32.
//   2. The sums, times the adapter's scale, become bf16 operands: two terms
//      (hi + lo, 16 bits) for bf16 outputs, whose own rounding is 2^-8, three
//      (24 bits) for fp32 outputs.
//   3. Up: each CTA takes tiles of 128 outputs.  B's rows come by TMA as they
//      lie in memory, the product goes to one of two TMEM buffers, and eight
//      warps turn it through shared memory so that base and y move in whole
//      32-byte sectors, a row's 32 outputs per four lanes.
//
// Bound: HBM.  base and y are 4 of the 5 bytes that an output costs at K =
// N / 2.7 and rank 64; the tensor work of 8192 x 2560 x 6912 at rank 64 (17
// GFLOP with two terms) is 9 us of the 41 us that its bytes take.
#include "bl_device.cuh"
#include "bl_internal.h"
#include "lora.cuh"

namespace bl {
namespace {

constexpr int kWarps = 10, kThreads = 32 * kWarps;  // TMA, MMA, 8 epilogue warps
constexpr int kEpilogue = 256;
constexpr int kStages = 3;                 // K blocks of 64 in flight
constexpr int kN = 128;                    // outputs of an up tile
constexpr uint32_t kXBytes = kTile * 128;  // 128 rows of 64 bf16
constexpr uint32_t kTmemCols = 256;        // two accumulators of 128 columns
constexpr int kTurn = 36;                  // floats of a row of 32 outputs being turned: 16-byte aligned, few conflicts

__host__ __device__ constexpr uint32_t idesc(int n) {  // bf16 x bf16 -> fp32, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
}

// Shared memory: [ring | operand terms + turning buffers][partial sums | up ring]
struct Plan {
  int rp, rk;             // rank rounded up to 16 (MMA N and K) and to 64 (operand sub-tiles)
  uint32_t a_bytes;       // of a ring stage's A block
  uint32_t stage;         // of a ring stage
  uint32_t term;          // of one operand term, [128][rk] in 64-column sub-tiles
  uint32_t turn_at;       // byte offset of the turning buffers
  uint32_t part_at;       // of the partial sums
  uint32_t part_row;      // floats of a row of them
  uint32_t up_stage;      // of an up tile of B
  uint32_t bar_at, total;
};
__host__ __device__ inline Plan make_plan(int rank, int terms) {
  Plan p;
  p.rp = (rank + 15) / 16 * 16;
  p.rk = (rank + 63) / 64 * 64;
  p.a_bytes = uint32_t(p.rp) * 128;
  p.stage = kXBytes + (p.a_bytes + 1023) / 1024 * 1024;
  p.term = uint32_t(p.rk) / 64 * kTile * 128;
  p.turn_at = p.term * terms;
  const uint32_t first = p.turn_at + 8 * 32 * kTurn * 4, ring = kStages * p.stage;
  p.part_at = ((first > ring ? first : ring) + 1023) / 1024 * 1024;
  p.part_row = uint32_t(p.rp) + 4;
  p.up_stage = uint32_t(p.rk) / 64 * kN * 128;
  const uint32_t part = kTile * p.part_row * 4;
  p.bar_at = p.part_at + (part > 2 * p.up_stage ? part : 2 * p.up_stage);
  p.total = p.bar_at + 256;
  return p;
}

struct Args {
  const int32_t* adapter;
  const float* scale;
  const void* base;
  void* y;
  unsigned int* err;
  int64_t M, N, K, L;
  int rank;
  bool vec;  // base and y rows are 16-byte aligned
};

struct Control {  // at Plan::bar_at
  uint64_t full[kStages], empty[kStages], sums[2], drained[2], up_full[2], up_empty[2], out_full[2], out_empty[2];
  uint32_t tmem, starts[4];
  int abort;
};
static_assert(sizeof(Control) <= 256, "");

// base[m, n .. n+8) as fp32; outputs past N are 0.
template <bool YB>
__device__ __forceinline__ void load_base(const Args& g, int64_t m, int n, float (&v)[8]) {
  const int64_t i = m * g.N + n;
  if (g.vec && n + 8 <= g.N) {
    load8<YB>(reinterpret_cast<const uint8_t*>(g.base) + i * (YB ? 2 : 4), 0, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = n + j < g.N ? load1<YB>(g.base, i + j) : 0.f;
}
template <bool YB>
__device__ __forceinline__ void store_y(const Args& g, int64_t m, int n, const float (&v)[8]) {
  const int64_t i = m * g.N + n;
  if (g.vec && n + 8 <= g.N) {
    store8<YB>(reinterpret_cast<uint8_t*>(g.y) + i * (YB ? 2 : 4), v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (n + j < g.N) store1<YB>(g.y, i + j, v[j]);
}

// The next run of the tile from token `t`: [t, end) and its adapter.
struct Runs {
  const uint32_t* starts;
  int t, end, size;
  __device__ __forceinline__ Runs(const uint32_t* s, int n) : starts(s), t(0), end(0), size(n) {}
  __device__ __forceinline__ bool next() {
    t = end;
    if (t >= size) return false;
    end = size;
    for (int w = (t + 1) / 32; w < 4; ++w) {
      uint32_t b = starts[w];
      if (w == (t + 1) / 32) b &= 0xFFFFFFFFu << ((t + 1) & 31);
      if (b) {
        end = min(size, w * 32 + __ffs(b) - 1);
        break;
      }
    }
    return true;
  }
};

template <int CL, bool YB>
__global__ void __launch_bounds__(kThreads) lora_tile_kernel(const __grid_constant__ CUtensorMap xmap,
                                                             const __grid_constant__ CUtensorMap amap,
                                                             const __grid_constant__ CUtensorMap bmap, const Args g) {
  constexpr int kTerms = YB ? 2 : 3;
  extern __shared__ __align__(1024) uint8_t smem[];
  const Plan p = make_plan(g.rank, kTerms);
  Control& c = *reinterpret_cast<Control*>(smem + p.bar_at);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t me = CL == 1 ? 0 : cluster_ctarank();
  const int64_t m0 = int64_t(blockIdx.x / CL) * kTile;
  const int size = int(min(int64_t(kTile), g.M - m0));
  volatile int* abort = &c.abort;

  if (warp == 1) {
    tmem_alloc(&c.tmem, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    c.abort = 0;
    for (int i = 0; i < kStages; ++i) mbar_init(&c.full[i], 1), mbar_init(&c.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.sums[i], 1);
      mbar_init(&c.drained[i], kEpilogue / 32);
      mbar_init(&c.up_full[i], 1);
      mbar_init(&c.up_empty[i], 1);
      mbar_init(&c.out_full[i], 1);
      mbar_init(&c.out_empty[i], kEpilogue / 32);
    }
    fence_barrier_init();
  }
  pdl_wait();
  if (threadIdx.x < kTile) {
    const int t = threadIdx.x;
    const int a = t < size ? adapter_of(g.adapter, m0 + t, g.L) : -1;
    const int before = t > 0 && t < size ? adapter_of(g.adapter, m0 + t - 1, g.L) : -2;
    const uint32_t b = __ballot_sync(0xffffffffu, t < size && a != before);
    if (lane == 0) c.starts[warp] = b;
    if (me == 0 && t < size && g.adapter[m0 + t] >= g.L && g.err) atomicOr(g.err, BL_DEVERR_RANGE);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  const bool mine = __popc(c.starts[0]) + __popc(c.starts[1]) + __popc(c.starts[2]) + __popc(c.starts[3]) <= kTileRuns;

  if (mine) {
    const int blocks = int((g.K + 63) / 64), per = (blocks + CL - 1) / CL;
    const int k0 = min(int(me) * per, blocks), k1 = min(k0 + per, blocks);
    // ---- 1. down ----
    if (warp == 0 && lane == 0) {
      int it = 0;
      for (Runs r(c.starts, size); r.next();) {
        const int a = adapter_of(g.adapter, m0 + r.t, g.L);
        if (a < 0) continue;
        for (int kb = k0; kb < k1; ++kb, ++it) {
          const int st = it % kStages;
          if (it >= kStages && !*abort && !mbar_wait_bounded(&c.empty[st], uint32_t(it / kStages - 1) & 1u, g.err))
            *abort = 1;
          if (*abort) break;
          mbar_arrive_expect_tx(&c.full[st], kXBytes + p.a_bytes);
          tma_load_2d(smem + st * p.stage, &xmap, kb * 128, int(m0), &c.full[st]);
          tma_load_2d(smem + st * p.stage + kXBytes, &amap, kb * 128, a * g.rank, &c.full[st]);
        }
        if (*abort) break;
      }
      // nothing may still be on its way into the ring when it is used for the operand
      for (int i = max(0, it - kStages); i < it; ++i)
        mbar_wait_bounded(&c.full[i % kStages], uint32_t(i / kStages) & 1u, nullptr);
    } else if (warp == 1 && lane == 0) {
      int it = 0, run = 0;
      const uint32_t sbase = smem_addr(smem);
      for (Runs r(c.starts, size); r.next();) {
        if (adapter_of(g.adapter, m0 + r.t, g.L) < 0) continue;
        const uint32_t acc = tmem + uint32_t(run & 1) * kN;
        if (run >= 2 && !*abort && !mbar_wait_bounded(&c.drained[run & 1], uint32_t(run / 2 - 1) & 1u, g.err)) *abort = 1;
        tc_fence_after();
        for (int kb = k0; kb < k1; ++kb, ++it) {
          const int st = it % kStages;
          if (!*abort && !mbar_wait_bounded(&c.full[st], uint32_t(it / kStages) & 1u, g.err)) *abort = 1;
          tc_fence_after();
          const uint32_t xa = sbase + st * p.stage, aa = xa + kXBytes;
          if (!*abort)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_f16(acc, umma_desc_sw128(xa + ks * 32), umma_desc_sw128(aa + ks * 32), idesc(p.rp), kb > k0 || ks > 0);
          umma_commit(&c.empty[st]);
        }
        umma_commit(&c.sums[run & 1]);
        ++run;
      }
    } else if (warp >= 2) {
      float* part = reinterpret_cast<float*>(smem + p.part_at);
      const int quarter = warp & 3, half = (warp - 2) >> 2, row = quarter * 32 + lane;
      int run = 0;
      for (Runs r(c.starts, size); r.next();) {
        if (adapter_of(g.adapter, m0 + r.t, g.L) < 0) continue;
        if (!*abort && !mbar_wait_bounded(&c.sums[run & 1], uint32_t(run / 2) & 1u, g.err)) *abort = 1;
        tc_fence_after();
        for (int col = half * 16; col < p.rp; col += 32) {
          uint32_t v[16];
          tmem_ld16(tmem + uint32_t(run & 1) * kN + (uint32_t(quarter * 32) << 16) + uint32_t(col), v);
          tmem_ld_wait();
          if (row >= r.t && row < r.end) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(part + row * p.part_row + col + 4 * j) =
                  k1 > k0 ? make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]) : make_uint4(0, 0, 0, 0);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.drained[run & 1]);
        ++run;
      }
    }
    tc_fence_before();
    __syncwarp();
    if (CL == 1) __syncthreads(); else cluster_sync();
    tc_fence_after();

    // ---- 2. the operand: eight columns of a row at a time ----
    for (int i = threadIdx.x; i < kTile * (p.rp / 8); i += kThreads) {
      const int row = i / (p.rp / 8), chunk = i % (p.rp / 8);
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const int a = row < size ? adapter_of(g.adapter, m0 + row, g.L) : -1;
      if (a >= 0 && chunk * 8 < g.rank) {
        const float* src = reinterpret_cast<const float*>(smem + p.part_at) + row * p.part_row + chunk * 8;
#pragma unroll
        for (int q = 0; q < CL; ++q) {
          const float4* f = reinterpret_cast<const float4*>(CL == 1 ? src : peer(src, q));
          const float4 f0 = f[0], f1 = f[1];
          v[0] += f0.x, v[1] += f0.y, v[2] += f0.z, v[3] += f0.w;
          v[4] += f1.x, v[5] += f1.y, v[6] += f1.z, v[7] += f1.w;
        }
        const float s = g.scale[a];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= s;
      }
      uint8_t* dst = smem + (chunk / 8) * (kTile * 128) + row * 128 + ((uint32_t(chunk & 7) ^ uint32_t(row & 7)) << 4);
#pragma unroll
      for (int t = 0; t < kTerms; ++t) {  // the nearest bf16, and the same of what it leaves
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = f32_to_bf16_bits_rn(v[2 * j]), hi = f32_to_bf16_bits_rn(v[2 * j + 1]);
          v[2 * j] -= bf16_bits_to_f32(uint16_t(lo));
          v[2 * j + 1] -= bf16_bits_to_f32(uint16_t(hi));
          w[j] = lo | hi << 16;
        }
        *reinterpret_cast<uint4*>(dst + t * p.term) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    fence_async_smem();
    if (CL == 1) __syncthreads(); else cluster_sync();  // and nobody reads the partial sums any more

    // ---- 3. up ----
    const int tiles = int((g.N + kN - 1) / kN);
    if (warp == 0 && lane == 0) {
      int it = 0;
      for (Runs r(c.starts, size); r.next();) {
        const int a = adapter_of(g.adapter, m0 + r.t, g.L);
        if (a < 0) continue;
        for (int n = int(me); n < tiles && !*abort; n += CL, ++it) {
          const int st = it & 1;
          if (it >= 2 && !mbar_wait_bounded(&c.up_empty[st], uint32_t(it / 2 - 1) & 1u, g.err)) {
            *abort = 1;
            break;
          }
          uint8_t* dst = smem + p.part_at + st * p.up_stage;
          mbar_arrive_expect_tx(&c.up_full[st], p.up_stage);
          for (int sub = 0; sub < p.rk / 64; ++sub)
            tma_load_2d(dst + sub * (kN * 128), &bmap, sub * 128, int(int64_t(a) * g.N + n * kN), &c.up_full[st]);
        }
      }
      // the CTA must not finish while a load still writes its shared memory
      for (int i = max(0, it - 2); i < it; ++i) mbar_wait_bounded(&c.up_full[i & 1], uint32_t(i / 2) & 1u, nullptr);
    } else if (warp == 1 && lane == 0) {
      int it = 0;
      const uint32_t sbase = smem_addr(smem);
      for (Runs r(c.starts, size); r.next();) {
        if (adapter_of(g.adapter, m0 + r.t, g.L) < 0) continue;
        for (int n = int(me); n < tiles; n += CL, ++it) {
          const int st = it & 1;
          if (!*abort && !mbar_wait_bounded(&c.up_full[st], uint32_t(it / 2) & 1u, g.err)) *abort = 1;
          if (it >= 2 && !*abort && !mbar_wait_bounded(&c.out_empty[st], uint32_t(it / 2 - 1) & 1u, g.err)) *abort = 1;
          tc_fence_after();
          const uint32_t ba = sbase + p.part_at + st * p.up_stage;
          if (!*abort)
            for (int t = 0; t < kTerms; ++t)
              for (int ks = 0; ks < p.rp / 16; ++ks) {
                const uint32_t off = uint32_t(ks >> 2) * (kTile * 128) + (ks & 3) * 32;
                umma_f16(tmem + st * kN, umma_desc_sw128(sbase + t * p.term + off), umma_desc_sw128(ba + off), idesc(kN),
                         t > 0 || ks > 0);
              }
          umma_commit(&c.up_empty[st]);
          umma_commit(&c.out_full[st]);
        }
      }
    } else if (warp >= 2) {
      const int quarter = warp & 3, half = (warp - 2) >> 2;
      float* turn = reinterpret_cast<float*>(smem + p.turn_at) + (warp - 2) * 32 * kTurn;
      int it = 0;
      for (Runs r(c.starts, size); r.next();) {
        const bool has = adapter_of(g.adapter, m0 + r.t, g.L) >= 0;
        // rows of this warp that are in the run
        const int ra = max(r.t, quarter * 32), rb = min(r.end, quarter * 32 + 32);
        if (!has) {
          if (g.y != g.base)
            for (int n = int(me) * kN + half * 64 + (lane & 7) * 8; n < int(g.N); n += CL * kN)
              for (int row = ra + (lane >> 3); row < rb; row += 4) {
                float v[8];
                load_base<YB>(g, m0 + row, n, v);
                store_y<YB>(g, m0 + row, n, v);
              }
          continue;
        }
        for (int n = int(me); n < tiles; n += CL, ++it) {
          const int st = it & 1, n0 = n * kN + half * 64 + (lane & 3) * 8;
          // base of the first 32 outputs, on its way while the product is formed
          float v[4][8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = quarter * 32 + 8 * i + (lane >> 2);
            if (row >= ra && row < rb && n0 < g.N) load_base<YB>(g, m0 + row, n0, v[i]);
          }
          if (!*abort && !mbar_wait_bounded(&c.out_full[st], uint32_t(it / 2) & 1u, g.err)) *abort = 1;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t d[32];
            const uint32_t at = tmem + st * kN + (uint32_t(quarter * 32) << 16) + uint32_t(half * 64 + h * 32);
            tmem_ld16(at, *reinterpret_cast<uint32_t(*)[16]>(d));
            tmem_ld16(at + 16, *reinterpret_cast<uint32_t(*)[16]>(d + 16));
            tmem_ld_wait();
            if (h == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&c.out_empty[st]);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(turn + lane * kTurn + 4 * j) =
                  make_uint4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]);
            __syncwarp();
            const int nn = n0 + h * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tr = 8 * i + (lane >> 2), row = quarter * 32 + tr;
              if (row < ra || row >= rb || nn >= g.N || *abort) continue;
              if (h == 1) load_base<YB>(g, m0 + row, nn, v[i]);
              const float4 f0 = *reinterpret_cast<const float4*>(turn + tr * kTurn + (lane & 3) * 8);
              const float4 f1 = *reinterpret_cast<const float4*>(turn + tr * kTurn + (lane & 3) * 8 + 4);
              v[i][0] += f0.x, v[i][1] += f0.y, v[i][2] += f0.z, v[i][3] += f0.w;
              v[i][4] += f1.x, v[i][5] += f1.y, v[i][6] += f1.z, v[i][7] += f1.w;
              store_y<YB>(g, m0 + row, nn, v[i]);
            }
          }
        }
      }
    }
  }
  __syncwarp();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int CL, bool YB>
cudaError_t launch_tiles(const CUtensorMap& xmap, const CUtensorMap& amap, const CUtensorMap& bmap, const Args& g,
                         cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint32_t smem = make_plan(g.rank, YB ? 2 : 3).total;
  const cudaError_t e = raise_smem_cap(lora_tile_kernel<CL, YB>, dev, int(make_plan(128, YB ? 2 : 3).total));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((g.M + kTile - 1) / kTile * CL));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (CL > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim = {CL, 1, 1};
    ++n;
  }
  if (overlap_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, lora_tile_kernel<CL, YB>, xmap, amap, bmap, g);
}

}  // namespace

cudaError_t launch_lora_tile(const void* x, const int32_t* adapter, const uint16_t* a, const uint16_t* b,
                             const float* scale, const void* base, void* y, bl_dtype yt, int64_t M, int64_t N,
                             int64_t K, int64_t adapters, int rank, cudaStream_t s) {
  CUtensorMap xmap, amap, bmap;  // bytes; 128-byte wide boxes, swizzled
  const Plan p = make_plan(rank, 2);
  if (adapters * rank > 0x7fffffff || adapters * N > 0x7fffffff || K * 2 > 0x7fffffff ||
      !encode_tmap_2d_u8(&xmap, x, uint64_t(K) * 2, uint64_t(M), uint64_t(K) * 2, 128, kTile, true) ||
      !encode_tmap_2d_u8(&amap, a, uint64_t(K) * 2, uint64_t(adapters * rank), uint64_t(K) * 2, 128, uint32_t(p.rp), true) ||
      !encode_tmap_2d_u8(&bmap, b, uint64_t(rank) * 2, uint64_t(adapters * N), uint64_t(rank) * 2, 128, kN, true))
    return cudaErrorNotSupported;
  const int es = yt == BL_BF16 ? 2 : 4;
  const bool vec = N * es % 16 == 0 && ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(y)) & 15) == 0;
  const Args g{adapter, scale, base, y, dev_error_ptr(), M, N, K, adapters, rank, vec};
  // CTAs of a tile: as many as keep two per SM busy
  const int64_t tiles = (M + kTile - 1) / kTile;
  int cl = 1;
  while (cl < 8 && tiles * cl * 2 <= 2 * sm_count()) cl *= 2;
  const bool yb = yt == BL_BF16;
  switch (cl) {
    case 1: return yb ? launch_tiles<1, true>(xmap, amap, bmap, g, s) : launch_tiles<1, false>(xmap, amap, bmap, g, s);
    case 2: return yb ? launch_tiles<2, true>(xmap, amap, bmap, g, s) : launch_tiles<2, false>(xmap, amap, bmap, g, s);
    case 4: return yb ? launch_tiles<4, true>(xmap, amap, bmap, g, s) : launch_tiles<4, false>(xmap, amap, bmap, g, s);
    default: return yb ? launch_tiles<8, true>(xmap, amap, bmap, g, s) : launch_tiles<8, false>(xmap, amap, bmap, g, s);
  }
}

}  // namespace bl
