// Low-rank adapters of long runs of tokens (bl_lora_add), on the 5th-generation
// tensor cores (tcgen05):
//   y[m,n] = base[m,n] + scale[a] * sum_r B[a,n,r] (sum_k A[a,r,k] x[m,k]).
//
// A cluster of CL CTAs takes 128 tokens; while there are few, several clusters
// do, each with the first product and a share of the outputs (512 tokens, 2560
// -> 6912, rank 64: 17 us).  A run is a stretch of those tokens
// with one adapter; a tile of more than kTileRuns runs is left to the kernel
// for scattered tokens.
//   1. Down: each CTA takes a part of K.  x (128 x 64 blocks) and the runs' A
//      (rank x 64, up to two runs at once) come by TMA through a ring; the
//      tensor core forms the 128 x rank product in TMEM.  It cuts its sums off
//      instead of rounding them, always towards zero: a bias of 1.8e-8 of the sum
//      for every 16 products of K, 1.6e-5 at K = 13824.  So the epilogue warps take
//      the sums over a few blocks (kChunk, kFloatChunk) and add them up in
//      registers, in fp32 to nearest, while the next ones are formed in a second
//      accumulator: 4e-7 at any K.  The rows of the run go to shared memory, and
//      the CTAs add their parts up in rank order through distributed shared memory.
//      fp32 x (two boxes of 32 columns) is turned by the epilogue warps into three
//      bf16 terms in TMEM, 24 bits (8192 tokens, 5120 -> 5120, rank 128: 116 us;
//      1894 on the CUDA cores; 112 if infinities were not looked for).
//   2. The sums, times the adapter's scale, become bf16 operands in TMEM, three
//      terms: 24 bits, as many as they have.  (With two, 16 bits, 0.2 % of the bf16
//      outputs were a step off; 8192 tokens, rank 64: 1 % less time, rank 128: 5 %.
//      In shared memory they would take up to 96 KB of what the rings have.)
//   3. Up: each CTA takes tiles of 256 bytes of outputs (128 bf16, 64 fp32).
//      B's rows come by TMA as they lie in memory, and so does the tile of
//      base, 128-byte swizzled, four in flight.  Every run of the 128 tokens
//      has its own product in one of two TMEM buffers; the thread of a row adds
//      its run's to the base in place, and the tile goes out by TMA, rows
//      without an adapter unchanged.  Rows of y that are not 16-byte aligned
//      (N * element size not a multiple of 16) are read and written by the
//      threads, a row's outputs by neighbouring lanes.
//
// A tile with several runs takes a product of each for every output tile, and
// so nearly twice as long; where SMs are left, a second cluster takes half of
// its outputs (12 % in the case below).
//
// Bound: HBM; base and y are 4 of the 5 bytes that an output costs at K = N / 2.7
// and rank 64.  8192 tokens of 12 prompts, 2560 -> 6912, rank 64: 58.7 us, 69 % of
// the copy rate for 276 MB, 13 us the tensor core's (24 GFLOP with three terms).
// One run's rows are not masked out of the other's product (one sum for both):
// an infinite weight of one request's adapter must not reach another's outputs.
#include <algorithm>

#include "bl_device.cuh"
#include "bl_internal.h"
#include "lora.cuh"

namespace bl {
namespace {

constexpr int kEpilogueWarps = 16;         // four per quarter of the TMEM lanes
constexpr int kWarps = 3 + kEpilogueWarps, kThreads = 32 * kWarps;  // x, A and B; MMA; epilogue; base and y
constexpr int kStages = 5;                 // K blocks of 64 in flight at most
constexpr int kFloatStages = 3;            // of fp32 x, whose terms take 96 TMEM columns each
constexpr int kUp = 6;                     // tiles of B in flight at most
constexpr int kMostHelped = 256;           // tiles of tokens among which helpers look for theirs
constexpr int kTiles = 4;                  // tiles of base in flight
constexpr uint32_t kXBytes = kTile * 128;  // 128 rows of 128 bytes: 64 bf16 of x; half a tile of base
constexpr int kAcc = 2, kAccCols = 128;    // accumulators
constexpr int kChunk = 4, kFloatChunk = 2; // blocks of K, of bf16 and fp32 x, whose sums the tensor core forms: 16 and 24 additions
constexpr int kTerms = 3;                  // of the operand
constexpr uint32_t kOperand = 256;         // TMEM column of its first term; a term takes 64 at most
constexpr uint32_t kTermsOfX = 128;        // TMEM column of the terms of fp32 x, three of 32 per stage
constexpr uint32_t kTmemCols = 512;
static_assert(kTermsOfX + kFloatStages * 96 <= kTmemCols, "");
constexpr int kTurn = 33;                  // floats of a row of 32 outputs being turned

__host__ __device__ constexpr uint32_t idesc(int n) {  // bf16 x bf16 -> fp32, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
}

// Shared memory.  First [ring of x and A | partial sums]; then, over both,
// [ring of B | ring of base, or turning buffers].
struct Plan {
  int rp, rk;             // rank rounded up to 16 (MMA N and K) and to 64 (operand sub-tiles)
  uint32_t a_bytes;       // of a run's A block in a ring stage
  int group;              // runs whose A goes through the ring together
  int stages, up;         // places of the ring of x and A, and of the ring of B
  uint32_t x_bytes;       // of a block of x: 64 bf16, or two halves of 32 floats, of 128 rows
  uint32_t stage;         // of a ring stage
  int term;               // TMEM columns of one operand term
  uint32_t part_at;       // byte offset of the partial sums
  uint32_t part_row;      // floats of a row of them
  uint32_t up_at, up_stage;  // ring of B tiles
  uint32_t base_at;       // ring of base tiles
  uint32_t end;
};
__host__ __device__ inline Plan make_plan(int rank, int n_tile, int runs, bool xf) {
  Plan p;
  p.rp = (rank + 15) / 16 * 16;
  p.rk = (rank + 63) / 64 * 64;
  p.a_bytes = uint32_t(p.rp) * 128;
  p.group = p.rp <= 64 && runs > 1 ? 2 : 1;
  p.x_bytes = xf ? 2 * kXBytes : kXBytes;
  p.stage = p.x_bytes + uint32_t(p.group) * p.a_bytes;
  p.stages = xf ? kFloatStages : p.rp <= 64 ? kStages : kStages - 1;
  p.term = p.rk / 2;
  p.up_at = 0;
  p.up_stage = uint32_t(p.rk) / 64 * n_tile * 128;
  p.up = p.rk == 64 ? kUp : kUp / 2;
  const uint32_t up_end = p.up_at + p.up * p.up_stage;
  p.part_at = p.stages * p.stage;
  p.part_row = uint32_t(p.rp) + 4;
  p.base_at = up_end;
  const uint32_t one = p.part_at + kTile * p.part_row * 4, two = p.base_at + kTiles * 2 * kXBytes;
  p.end = ((one > two ? one : two) + 1023) / 1024 * 1024;
  return p;
}

// The control block lies behind either layout.
__host__ __device__ inline uint32_t control_at(int rank, int n_tile, bool xf) {
  const uint32_t one = make_plan(rank, n_tile, 1, xf).end, two = make_plan(rank, n_tile, 2, xf).end;
  return one > two ? one : two;
}

// A place in a ring of `n`, and how often it has gone round (a division by a
// number known at run time costs a few hundred clocks in a one-lane loop).
struct Ring {
  int n, at, round;
  __device__ __forceinline__ explicit Ring(int size) : n(size), at(0), round(0) {}
  __device__ __forceinline__ void next() {
    if (++at == n) at = 0, ++round;
  }
  __device__ __forceinline__ uint32_t parity() const { return uint32_t(round) & 1u; }           // of a wait for data
  __device__ __forceinline__ uint32_t free_parity() const { return uint32_t(round - 1) & 1u; }  // of a wait for room
};

struct Args {
  const int32_t* adapter;
  const float* scale;
  const void* base;
  void* y;
  unsigned int* err;
  int64_t M, N, K, L;
  int rank;
  bool xf;     // x is fp32
  int shares;  // clusters of 128 tokens: each forms the inner products, and a share of the outputs
  int tiles;   // of 128 tokens
  int helpers; // clusters beyond tiles * shares: each takes half of the outputs of a tile with several runs
};

struct Control {  // at control_at()
  uint64_t full[kStages], empty[kStages], terms[kFloatStages], sums[kAcc], drained[kAcc], up_full[kUp], up_empty[kUp], out_full[kAcc], out_empty[kAcc];
  uint64_t base_full[kTiles], base_done[kTiles];
  uint32_t tmem, starts[4], used[4];  // used: runs that have an adapter
  uint32_t several[kMostHelped / 32]; // bit t: tile t has several runs, and is this kernel's
  int abort;
  int adapter[kTile];  // of each token, -1: none
};
static_assert(sizeof(Control) <= 1024, "");

// The runs of a tile, at most kTileRuns, in registers: eight bits for each
// end, a bit for each that has an adapter.
struct RunTable {
  uint64_t ends;
  uint32_t has;
  int n;
  __device__ __forceinline__ RunTable(const uint32_t* starts, const int* adapter, int size) : ends(0), has(0), n(0) {
    for (int w = 0; w < kTile / 32; ++w)
      for (uint32_t bits = starts[w]; bits && n < kTileRuns; bits &= bits - 1) {
        const int t = w * 32 + __ffs(bits) - 1;
        if (n > 0) ends |= uint64_t(t) << (8 * (n - 1));
        has |= uint32_t(adapter[t] >= 0) << n;
        ++n;
      }
    ends |= uint64_t(size) << (8 * (n - 1));
  }
};

// A walk over them: tokens [t, end).
struct Runs {
  const RunTable& table;
  int i, t, end;
  __device__ __forceinline__ explicit Runs(const RunTable& r) : table(r), i(0), t(0), end(0) {}
  __device__ __forceinline__ bool next() {
    if (i == table.n) return false;
    t = end;
    end = int(table.ends >> (8 * i)) & 255;
    ++i;
    return true;
  }
  __device__ __forceinline__ bool has() const { return (table.has >> (i - 1)) & 1u; }
  // The next `most` (one or two) runs with an adapter: their tokens [t[j], end[j]).
  __device__ __forceinline__ int group(int most, int (&from)[2], int (&to)[2]) {
    int n = 0;
    while (n < most && next())
      if (has()) {
        if (n == 0)
          from[0] = t, to[0] = end;
        else
          from[1] = t, to[1] = end;
        ++n;
      }
    return n;
  }
};

// Whether the condition holds in every lane.  Each lane polls a barrier by
// itself, and tcgen05.ld is undefined unless the whole warp executes it
// together: a warp-wide vote after the wait brings the lanes together again and
// gives them one decision (the flag may be raised between two lanes' reads).
__device__ __forceinline__ bool warp_agrees(bool c) { return __all_sync(0xffffffffu, c) != 0; }

// Two bf16, infinities turned into the largest finite ones.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tmin.bf16x2 t, %1, %2;\n\tmax.bf16x2 %0, t, %3;\n\t}"
      : "=r"(r)
      : "r"(w), "r"(0x7f7f7f7fu), "r"(0xff7fff7fu));
  return r;
}

// The bf16 nearest to each of v, two at a time, as term t; v keeps what they leave.  What rounds to an infinity takes
// the largest bf16 as its first term, so that a finite value stays finite; an infinity is left over as itself, and is
// every later term (never inf - inf).
template <int N>
__device__ __forceinline__ void take_term(float (&v)[N], uint32_t (&w)[N / 2], int t) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    w[j] = bf16x2_rn(v[2 * j], v[2 * j + 1]);
    const uint32_t f = finite_bf16x2(w[j]);
    if (t == 0) w[j] = f;
    v[2 * j] -= __uint_as_float(f << 16);
    v[2 * j + 1] -= __uint_as_float(f & 0xffff0000u);
  }
}

// The tiles of tokens with several runs, at most kTileRuns (a warp a tile at a time), by the whole CTA.
__device__ __forceinline__ void find_several(const Args& g, uint32_t (&several)[kMostHelped / 32]) {
  const int lane = threadIdx.x & 31;
  __syncthreads();
  if (threadIdx.x < kMostHelped / 32) several[threadIdx.x] = 0;
  __syncthreads();
  for (int tile = threadIdx.x >> 5; tile < g.tiles; tile += kWarps) {
    int starts = 0, used = 0;
#pragma unroll
    for (int j = 0; j < kTile / 32; ++j) {
      const int64_t t = int64_t(tile) * kTile + 32 * j + lane;
      const int a = t < g.M ? adapter_of(g.adapter, t, g.L) : -1;
      const int before = t < g.M && (j > 0 || lane > 0) ? adapter_of(g.adapter, t - 1, g.L) : -2;
      const uint32_t start = __ballot_sync(0xffffffffu, t < g.M && a != before);
      starts += __popc(start);
      used += __popc(start & __ballot_sync(0xffffffffu, a >= 0));
    }
    if (lane == 0 && used > 1 && starts <= kTileRuns) atomicOr(&several[tile >> 5], 1u << (tile & 31));
  }
  __syncthreads();
}

// YB: base and y are bf16.  TMA: they come and go by TMA.
template <int CL, bool YB, bool TMA>
__global__ void __launch_bounds__(kThreads, 1) lora_tile_kernel(const __grid_constant__ CUtensorMap xmap,
                                                             const __grid_constant__ CUtensorMap amap,
                                                             const __grid_constant__ CUtensorMap bmap,
                                                             const __grid_constant__ CUtensorMap base_map,
                                                             const __grid_constant__ CUtensorMap y_map, const Args g) {
  const int chunk = g.xf ? kFloatChunk : kChunk;
  constexpr int kN = YB ? 128 : 64;  // outputs of an up tile
  constexpr int kHalf = kN / 2;      // 128 bytes of them
  extern __shared__ __align__(1024) uint8_t smem[];
  Control& c = *reinterpret_cast<Control*>(smem + control_at(g.rank, kN, g.xf));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t me = CL == 1 ? 0 : cluster_ctarank();
  const int cluster = int(blockIdx.x / CL), helper = cluster - g.tiles * g.shares;  // helper >= 0: one of them
  volatile int* abort = &c.abort;

  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&c.tmem, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    c.abort = 0;
    for (int i = 0; i < kStages; ++i) mbar_init(&c.full[i], 1), mbar_init(&c.empty[i], 1);
    for (int i = 0; i < kFloatStages; ++i) mbar_init(&c.terms[i], kEpilogueWarps);
    for (int i = 0; i < kUp; ++i) mbar_init(&c.up_full[i], 1), mbar_init(&c.up_empty[i], 1);
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&c.sums[i], 1);
      mbar_init(&c.drained[i], kEpilogueWarps);
      mbar_init(&c.out_full[i], 1);
      mbar_init(&c.out_empty[i], kEpilogueWarps);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&c.base_full[i], 1);
      mbar_init(&c.base_done[i], kEpilogueWarps);
    }
    fence_barrier_init();
  }
  pdl_wait();
  int tile = cluster / g.shares;
  int first = cluster % g.shares * CL + int(me), step = g.shares * CL;  // of this CTA's tiles of outputs
  bool idle = false;
  if (helper >= 0) {  // the helper-th tile of several runs
    find_several(g, c.several);
    int left = helper;
    tile = -1;
    for (int w = 0; w < kMostHelped / 32 && tile < 0; ++w) {
      uint32_t bits = c.several[w];
      if (left >= __popc(bits)) {
        left -= __popc(bits);
        continue;
      }
      for (; left > 0; --left) bits &= bits - 1;
      tile = w * 32 + __ffs(bits) - 1;
    }
    idle = tile < 0;
    tile = max(tile, 0);
    first = CL + int(me), step = 2 * CL;
  }
  const int64_t m0 = int64_t(tile) * kTile;
  const int size = int(min(int64_t(kTile), g.M - m0));
  if (threadIdx.x < kTile) {
    const int t = threadIdx.x;
    const int a = t < size ? adapter_of(g.adapter, m0 + t, g.L) : -1;
    c.adapter[t] = a;
    const int before = t > 0 && t < size ? adapter_of(g.adapter, m0 + t - 1, g.L) : -2;
    const uint32_t b = __ballot_sync(0xffffffffu, t < size && a != before);
    const uint32_t u = __ballot_sync(0xffffffffu, t < size && a != before && a >= 0);
    if (lane == 0) c.starts[warp] = b, c.used[warp] = u;
    if (me == 0 && first < CL && t < size && g.adapter[m0 + t] >= g.L && g.err) atomicOr(g.err, BL_DEVERR_RANGE);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  const int starts = __popc(c.starts[0]) + __popc(c.starts[1]) + __popc(c.starts[2]) + __popc(c.starts[3]);
  const bool mine = starts <= kTileRuns && !idle;
  const RunTable table(c.starts, c.adapter, size);
  if (g.helpers > 0 && helper < 0 && mine && __popc(table.has) > 1) {  // does it have a helper?
    find_several(g, c.several);
    int before = 0;
    for (int w = 0; w < tile / 32; ++w) before += __popc(c.several[w]);
    before += __popc(c.several[tile / 32] & ((1u << (tile & 31)) - 1));
    if (before < g.helpers) step = 2 * CL;
  }

  if (warp == 2 + kEpilogueWarps && lane == 0) {  // it has nothing else to do yet
    // The kernel for the other tiles starts here and ends after this one.  It does not wait for the grids before, whose
    // results this grid's wait has made visible to this grid's threads: the fence passes them on.
    __threadfence();
    pdl_launch_dependents();
  }
  const Plan p = make_plan(g.rank, kN, __popc(c.used[0]) + __popc(c.used[1]) + __popc(c.used[2]) + __popc(c.used[3]), g.xf);

  // All threads of the cluster; the barrier wants converged warps.
  auto sync_all = [] {
    __syncwarp();
    if (CL == 1)
      __syncthreads();
    else
      cluster_sync();
  };

  if (mine) {
    const int blocks = int((g.K + 63) / 64), per = (blocks + CL - 1) / CL;
    const int k0 = min(int(me) * per, blocks), k1 = min(k0 + per, blocks);
    const int tiles = int((g.N + kN - 1) / kN);
    // TMEM beside the first accumulator: the terms of fp32 x, of three blocks or two, and the second accumulator
    const int term_sets = p.group * p.rp <= int(kTmemCols - kTermsOfX - kFloatStages * 96) ? kFloatStages : kFloatStages - 1;
    const uint32_t second = g.xf ? kTermsOfX + uint32_t(term_sets) * 96 : kAccCols;
    // ---- 1. down ----
    // Runs with an adapter, in groups whose A blocks go through the ring beside one block of x.
    if (warp == 0 && elect_one()) {
      Ring at(p.stages);
      Runs r(table);
      for (int from[2], to[2], n; (n = r.group(p.group, from, to)) > 0 && !*abort;) {
        for (int kb = k0; kb < k1; ++kb, at.next()) {
          const int st = at.at;
          if (at.round > 0 && !*abort && !mbar_wait_bounded(&c.empty[st], at.free_parity(), g.err)) *abort = 1;
          if (*abort) break;
          uint8_t* dst = smem + st * p.stage;
          mbar_arrive_expect_tx(&c.full[st], p.x_bytes + n * p.a_bytes);
          tma_load_2d(dst, &xmap, kb * int(p.x_bytes / kTile), int(m0), &c.full[st]);
          if (g.xf) tma_load_2d(dst + kXBytes, &xmap, kb * 256 + 128, int(m0), &c.full[st]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (j < n) tma_load_2d(dst + p.x_bytes + j * p.a_bytes, &amap, kb * 128, c.adapter[from[j]] * g.rank, &c.full[st]);
        }
      }
      // nothing may still be on its way into the ring when it is used for the operand
      for (int st = 0; st < p.stages; ++st)  // the last use of each place
        if (at.round > 0 || st < at.at)
          mbar_wait_bounded(&c.full[st], uint32_t(st < at.at ? at.round : at.round - 1) & 1u, nullptr);
    } else if (warp == 1 && elect_one()) {
      Ring at(p.stages), terms(term_sets), sum(kAcc);
      const uint32_t sbase = smem_addr(smem);
      Runs r(table);
      for (int from[2], to[2], n; (n = r.group(p.group, from, to)) > 0;)
        for (int kb = k0; kb < k1; sum.next()) {
          if (sum.round > 0 && !*abort && !mbar_wait_bounded(&c.drained[sum.at], sum.free_parity(), g.err)) *abort = 1;
          tc_fence_after();
          const uint32_t da = tmem + uint32_t(sum.at) * second;
          for (const int first_kb = kb, end = min(kb + chunk, k1); kb < end; ++kb, at.next(), terms.next()) {
            const int st = at.at;
            if (!*abort && !mbar_wait_bounded(&c.full[st], at.parity(), g.err)) *abort = 1;
            tc_fence_after();
            const uint32_t xa = sbase + st * p.stage;
            // the runs' A blocks lie one behind the other: one product for all
            if (g.xf) {
              if (!*abort && !mbar_wait_bounded(&c.terms[terms.at], terms.parity(), g.err)) *abort = 1;
              tc_fence_after();
              if (!*abort)
                for (int t = 2; t >= 0; --t)  // the smallest first, as in the second product
#pragma unroll
                  for (int ks = 0; ks < 4; ++ks)
                    umma_f16_ta(da, tmem + kTermsOfX + uint32_t(terms.at * 96 + t * 32 + ks * 8),
                                umma_desc_sw128(xa + p.x_bytes + ks * 32), idesc(n * p.rp), kb > first_kb || t < 2 || ks > 0);
            } else if (!*abort) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                umma_f16(da, umma_desc_sw128(xa + ks * 32), umma_desc_sw128(xa + kXBytes + ks * 32), idesc(n * p.rp),
                         kb > first_kb || ks > 0);
            }
            umma_commit(&c.empty[st]);
          }
          umma_commit(&c.sums[sum.at]);
        }
    } else if (warp >= 2 && warp < 2 + kEpilogueWarps) {
      float* part = reinterpret_cast<float*>(smem + p.part_at);
      const int quarter = warp & 3, part4 = (warp - 2) >> 2, row = quarter * 32 + lane;
      Ring at(p.stages), terms(term_sets), used(p.stages), sum(kAcc);
      // the terms of x, 16 columns of a row in a thread: unit u of a 128-byte row is at u ^ (row % 8)
      auto make_terms = [&] {
        const int st = at.at;
        if (!*abort && !mbar_wait_bounded(&c.full[st], at.parity(), g.err)) *abort = 1;
        if (terms.round > 0) {  // the products with the terms that were there
          if (!*abort && !mbar_wait_bounded(&c.empty[used.at], used.parity(), g.err)) *abort = 1;
          used.next();
        }
        tc_fence_after();
        float v[16];
        const uint8_t* mine_row = smem + st * p.stage + (part4 >> 1) * kXBytes + row * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 f = *reinterpret_cast<const float4*>(mine_row + (((part4 & 1) * 4 + u) ^ (row & 7)) * 16);
          v[4 * u] = f.x, v[4 * u + 1] = f.y, v[4 * u + 2] = f.z, v[4 * u + 3] = f.w;
        }
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          uint32_t w[8];
          take_term(v, w, t);
          __syncwarp();
          tmem_st8(tmem + kTermsOfX + uint32_t(terms.at * 96 + t * 32 + part4 * 8) + (uint32_t(quarter * 32) << 16), w);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.terms[terms.at]);
        at.next(), terms.next();
      };
      Runs r(table);
      for (int from[2], to[2], n; (n = r.group(p.group, from, to)) > 0;) {
        // two pieces of 16 columns: of each run's, or of the one's
        float total[2][16] = {};
        int col[2], begin[2], end[2];
        bool here[2];  // the warp has rows of the run
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool other = i > 0 && p.rp <= 64;
          col[i] = part4 * 16 + (i > 0 && !other ? 64 : 0);
          begin[i] = other ? from[1] : from[0], end[i] = other ? to[1] : to[0];
          here[i] = (!other || n > 1) && col[i] < p.rp && max(begin[i], quarter * 32) < min(end[i], quarter * 32 + 32);
        }
        int ready = k0;  // blocks whose terms are made
        for (int kb = k0; kb < k1; kb += chunk, sum.next()) {
          if (g.xf)  // those of the next sums before these are waited for
            for (; ready < min(kb + 2 * chunk, k1); ++ready) make_terms();
          if (!*abort && !mbar_wait_bounded(&c.sums[sum.at], sum.parity(), g.err)) *abort = 1;
          tc_fence_after();
          if (warp_agrees(!*abort)) {  // and the warp is converged for tcgen05.ld
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!here[i]) continue;
              uint32_t v[16];
              __syncwarp();
              tmem_ld16(tmem + uint32_t(sum.at) * second + uint32_t((i > 0 && p.rp <= 64 ? p.rp : 0) + col[i]) + (uint32_t(quarter * 32) << 16), v);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 16; ++q) total[i][q] += __uint_as_float(v[q]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.drained[sum.at]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (here[i] && row >= begin[i] && row < end[i]) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<float4*>(part + row * p.part_row + col[i] + 4 * q) =
                  make_float4(total[i][4 * q], total[i][4 * q + 1], total[i][4 * q + 2], total[i][4 * q + 3]);
          }
      }
    }
    tc_fence_before();
    sync_all();
    tc_fence_after();

    // ---- 2. the operand ----
    // A CTA adds up its rows of all parts, in rank order, and gives the sums to all (each reading all parts
    // itself, a row in a thread, took 35 us in clusters of 8 at rank 64).
    if (CL > 1) {
      constexpr int kRows = kTile / CL;
      const int quads = p.rp / 4;
      for (int i = threadIdx.x; i < kRows * quads; i += kThreads) {
        float* at = reinterpret_cast<float*>(smem + p.part_at) + (int(me) * kRows + i / quads) * p.part_row + i % quads * 4;
        float4 f[CL];
#pragma unroll
        for (int q = 0; q < CL; ++q) f[q] = *reinterpret_cast<const float4*>(peer(at, q));
#pragma unroll
        for (int q = 1; q < CL; ++q) f[0].x += f[q].x, f[0].y += f[q].y, f[0].z += f[q].z, f[0].w += f[q].w;
#pragma unroll
        for (int q = 0; q < CL; ++q) *reinterpret_cast<float4*>(peer(at, q)) = f[0];
      }
      sync_all();
    }
    // then a thread 32 columns of a row at a time
    if (warp >= 2 && warp < 2 + kEpilogueWarps) {
      const int quarter = warp & 3, part4 = (warp - 2) >> 2, row = quarter * 32 + lane;
      const int a = c.adapter[row];
      const float scale = a >= 0 ? g.scale[a] : 0.f;
      for (int k = part4 * 32; k < p.rk; k += 128) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
        if (a >= 0) {
          const float4* f = reinterpret_cast<const float4*>(smem + p.part_at) + (row * p.part_row + k) / 4;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (k + 4 * j < g.rank) {
              const float4 f4 = f[j];
              v[4 * j] = f4.x * scale, v[4 * j + 1] = f4.y * scale, v[4 * j + 2] = f4.z * scale, v[4 * j + 3] = f4.w * scale;
            }
        }
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {  // the nearest bf16, and the same of what it leaves
          uint32_t w[16];
          take_term(v, w, t);
          __syncwarp();
          tmem_st16(tmem + kOperand + uint32_t(t * p.term + k / 2) + (uint32_t(quarter * 32) << 16), w);
        }
      }
      __syncwarp();
      tmem_st_wait();
    }
    tc_fence_before();
    fence_async_smem();  // the rings come over the partial sums
    __syncthreads();  // and nobody reads the partial sums any more
    tc_fence_after();

    // ---- 3. up ----
    if (warp == 0 && elect_one()) {
      Ring at(p.up);
      for (int n = first; n < tiles && !*abort; n += step) {
        for (Runs r(table); r.next();) {
          if (!r.has()) continue;
          const int a = c.adapter[r.t];
          const int st = at.at;
          if (at.round > 0 && !mbar_wait_bounded(&c.up_empty[st], at.free_parity(), g.err)) {
            *abort = 1;
            break;
          }
          uint8_t* dst = smem + p.up_at + st * p.up_stage;
          mbar_arrive_expect_tx(&c.up_full[st], p.up_stage);
          for (int sub = 0; sub < p.rk / 64; ++sub)
            tma_load_2d(dst + sub * (kN * 128), &bmap, sub * 128, int(int64_t(a) * g.N + n * kN), &c.up_full[st]);
          at.next();
        }
      }
      // the CTA must not finish while a load still writes its shared memory
      for (int st = 0; st < p.up; ++st)
        if (at.round > 0 || st < at.at)
          mbar_wait_bounded(&c.up_full[st], uint32_t(st < at.at ? at.round : at.round - 1) & 1u, nullptr);
    } else if (warp == 1 && elect_one()) {
      // a product for every tile and run with an adapter, in the order in which B comes
      const int products = (tiles - first + step - 1) / step * __popc(table.has);
      const uint32_t sbase = smem_addr(smem);
      bool dead = *abort;
      Ring at(p.up);
      for (int it = 0; it < products; ++it, at.next()) {
        const int st = at.at, acc = it % kAcc;
        dead = dead || !mbar_wait_bounded(&c.up_full[st], at.parity(), g.err);
        dead = dead || (it >= kAcc && !mbar_wait_bounded(&c.out_empty[acc], uint32_t(it / kAcc - 1) & 1u, g.err));
        if (dead) *abort = 1;
        tc_fence_after();
        // 16 columns of the operand and of B's rows at a time (8 TMEM columns, 32 bytes), 64 where there
        // are so many: one descriptor after the other is made while the tensor core works
        const uint32_t ba = sbase + p.up_at + st * p.up_stage, da = tmem + acc * kAccCols;
        if (!dead)
          for (int t = kTerms - 1; t >= 0; --t)  // the smallest first: an addition drops bits below the sum's own
            for (int sub = 0; sub < p.rk / 64; ++sub) {
              const uint32_t oa = tmem + kOperand + uint32_t(t * p.term + 32 * sub), bs = ba + sub * (kN * 128);
              const uint32_t more = t < kTerms - 1 || sub > 0;
              if (p.rp - 64 * sub >= 64) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  umma_f16_ta(da, oa + 8 * ks, umma_desc_sw128(bs + ks * 32), idesc(kN), ks > 0 ? 1u : more);
              } else {
                for (int ks = 0; ks < p.rp / 16 - 4 * sub; ++ks)
                  umma_f16_ta(da, oa + 8 * ks, umma_desc_sw128(bs + ks * 32), idesc(kN), ks > 0 ? 1u : more);
              }
            }
        umma_commit(&c.up_empty[st]);
        umma_commit(&c.out_full[acc]);
      }
      if (dead && products > 0)  // none may still run when the CTA ends
        mbar_wait_bounded(&c.out_full[(products - 1) % kAcc], uint32_t((products - 1) / kAcc) & 1u, nullptr);
    } else if (warp >= 2 && warp < 2 + kEpilogueWarps) {
      constexpr int kCols = kN / 4;  // outputs of a warp: 64 bytes of a row
      const int quarter = warp & 3, part4 = (warp - 2) >> 2, row = quarter * 32 + lane;
      float* turn = reinterpret_cast<float*>(smem + p.base_at) + (warp - 2) * 32 * kTurn;
      int it = 0, tl = 0;
      for (int n = first; n < tiles; n += step, ++tl) {
        const int bs = tl % kTiles, n0 = n * kN + part4 * kCols;
        // this thread's 64 bytes of base: 16-byte unit u of a 128-byte row at u ^ (row % 8)
        uint8_t* mine_row = smem + p.base_at + (bs * 2 + (part4 >> 1)) * kXBytes + row * 128;
        auto unit = [&](int u) { return reinterpret_cast<uint4*>(mine_row + (((part4 & 1) * 4 + u) ^ (row & 7)) * 16); };
        if (TMA && !*abort && !mbar_wait_bounded(&c.base_full[bs], uint32_t(tl / kTiles) & 1u, g.err)) *abort = 1;
        for (Runs r(table); r.next();) {
          // rows of this warp that are in the run
          const int ra = max(r.t, quarter * 32), rb = min(r.end, quarter * 32 + 32);
          if (!r.has()) {
            if (!TMA && g.y != g.base)
              for (int i = ra + lane / kCols; i < rb; i += 32 / kCols) {
                const int j = n0 + lane % kCols;
                if (j < g.N) store1<YB>(g.y, (m0 + i) * g.N + j, load1<YB>(g.base, (m0 + i) * g.N + j));
              }
            continue;
          }
          const int acc = it % kAcc;
          if (!*abort && !mbar_wait_bounded(&c.out_full[acc], uint32_t(it / kAcc) & 1u, g.err)) *abort = 1;
          tc_fence_after();
          const bool ok = warp_agrees(!*abort);  // and the warp is converged for tcgen05.ld
          if (ra < rb && ok && n0 < g.N) {
            const uint32_t at = tmem + acc * kAccCols + (uint32_t(quarter * 32) << 16) + uint32_t(part4 * kCols);
            uint32_t d[kCols];
            __syncwarp();
#pragma unroll
            for (int h = 0; h < kCols; h += 16) tmem_ld16(at + h, *reinterpret_cast<uint32_t(*)[16]>(d + h));
            if (TMA) {
              uint4 v[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) v[u] = *unit(u);
              tmem_ld_wait();
              if (row >= ra && row < rb) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    w[j] = YB ? bf16x2_rn(__uint_as_float(w[j] << 16) + __uint_as_float(d[(8 * u + 2 * j) % kCols]),
                                          __uint_as_float(w[j] & 0xffff0000u) + __uint_as_float(d[(8 * u + 2 * j + 1) % kCols]))
                              : __float_as_uint(__uint_as_float(w[j]) + __uint_as_float(d[(4 * u + j) % kCols]));
                  *unit(u) = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            } else {
              tmem_ld_wait();
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kCols; ++j) turn[lane * kTurn + j] = __uint_as_float(d[j]);
              __syncwarp();
              const int nn = n0 + lane % kCols;
              constexpr int kStep = 32 / kCols;  // rows at a time
              if (nn < g.N)
                for (int i = ra + lane / kCols; i < rb; i += 8 * kStep) {
                  float v[8];
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    if (i + j * kStep < rb) v[j] = load1<YB>(g.base, (m0 + i + j * kStep) * g.N + nn);
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    if (i + j * kStep < rb)
                      store1<YB>(g.y, (m0 + i + j * kStep) * g.N + nn,
                                 v[j] + turn[(i + j * kStep - quarter * 32) * kTurn + lane % kCols]);
                }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.out_empty[acc]);
          ++it;
        }
        if (TMA) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.base_done[bs]);
        }
      }
    } else if (TMA && warp == 2 + kEpilogueWarps && elect_one()) {
      auto fetch = [&](int n, int bs) {
        const bool two = int64_t(n) * kN + kHalf < g.N;
        uint8_t* dst = smem + p.base_at + bs * 2 * kXBytes;
        mbar_arrive_expect_tx(&c.base_full[bs], two ? 2 * kXBytes : kXBytes);
        tma_load_2d(dst, &base_map, n * 256, int(m0), &c.base_full[bs]);
        if (two) tma_load_2d(dst + kXBytes, &base_map, n * 256 + 128, int(m0), &c.base_full[bs]);
      };
      int tl = 0, asked = 0;  // tiles stored, tiles asked for
      for (; asked < kTiles && first + asked * step < tiles; ++asked) fetch(first + asked * step, asked);
      for (int n = first; n < tiles; n += step, ++tl) {
        const int bs = tl % kTiles;
        if (!*abort && !mbar_wait_bounded(&c.base_done[bs], uint32_t(tl / kTiles) & 1u, g.err)) *abort = 1;
        if (*abort) break;
        const uint8_t* src = smem + p.base_at + bs * 2 * kXBytes;
        tma_store_2d(&y_map, n * 256, int(m0), src);
        if (int64_t(n) * kN + kHalf < g.N) tma_store_2d(&y_map, n * 256 + 128, int(m0), src + kXBytes);
        bulk_commit();
        bulk_wait_read();
        if (n + kTiles * step < tiles) fetch(n + kTiles * step, bs), ++asked;
      }
      // the CTA must not finish while a load still writes its shared memory
      for (int i = max(0, asked - kTiles); i < asked; ++i)
        mbar_wait_bounded(&c.base_full[i % kTiles], uint32_t(i / kTiles) & 1u, nullptr);
      bulk_wait();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

struct Maps {
  CUtensorMap x, a, b, base, y;
};

template <int CL, bool YB, bool TMA>
cudaError_t launch_tiles(const Maps& maps, const Args& g, cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  constexpr int kN = YB ? 128 : 64;
  const cudaError_t e = raise_smem_cap(lora_tile_kernel<CL, YB, TMA>, dev, int(std::max(control_at(128, kN, false), control_at(128, kN, true)) + 1024));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(g.tiles) * g.shares + g.helpers) * CL));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = control_at(g.rank, kN, g.xf) + 1024;
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
  return cudaLaunchKernelEx(&cfg, lora_tile_kernel<CL, YB, TMA>, maps.x, maps.a, maps.b, maps.base, maps.y, g);
}

template <bool YB, bool TMA>
cudaError_t launch_tiles(int cl, const Maps& maps, const Args& g, cudaStream_t s) {
  switch (cl) {
    case 1: return launch_tiles<1, YB, TMA>(maps, g, s);
    case 2: return launch_tiles<2, YB, TMA>(maps, g, s);
    case 4: return launch_tiles<4, YB, TMA>(maps, g, s);
    default: return launch_tiles<8, YB, TMA>(maps, g, s);
  }
}

}  // namespace

cudaError_t launch_lora_tile(const void* x, bl_dtype xt, const int32_t* adapter, const uint16_t* a, const uint16_t* b,
                             const float* scale, const void* base, void* y, bl_dtype yt, int64_t M, int64_t N,
                             int64_t K, int64_t adapters, int rank, cudaStream_t s) {
  const bool yb = yt == BL_BF16;
  const bool xf = xt == BL_F32;
  const uint64_t row = uint64_t(N) * (yb ? 2 : 4), x_row = uint64_t(K) * (xf ? 4 : 2);
  Maps maps;  // bytes; 128-byte wide boxes, swizzled
  if (adapters * rank > 0x7fffffff || adapters * N > 0x7fffffff || row > 0x7fffffff ||
      !encode_tmap_2d_u8(&maps.x, x, x_row, uint64_t(M), x_row, 128, kTile, true) ||
      !encode_tmap_2d_u8(&maps.a, a, uint64_t(K) * 2, uint64_t(adapters * rank), uint64_t(K) * 2, 128,
                         uint32_t(rank + 15) / 16 * 16, true) ||
      !encode_tmap_2d_u8(&maps.b, b, uint64_t(rank) * 2, uint64_t(adapters * N), uint64_t(rank) * 2, 128, yb ? 128 : 64,
                         true))
    return cudaErrorNotSupported;
  const bool tma = row % 16 == 0 && ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(y)) & 15) == 0 &&
                   encode_tmap_2d_u8(&maps.base, base, row, uint64_t(M), row, 128, kTile, true) &&
                   encode_tmap_2d_u8(&maps.y, y, row, uint64_t(M), row, 128, kTile, true);
  if (!tma) maps.base = maps.y = maps.x;  // not used
  Args g{adapter, scale, base, y, dev_error_ptr(), M, N, K, adapters, rank, xf, 1, 0, 0};
  // CTAs of a tile of tokens: as many as run at once
  const int64_t tiles = (M + kTile - 1) / kTile;
  int cl = 1;
  while (cl < 8 && tiles <= clusters_at_once(2 * cl)) cl *= 2;
  // and clusters of them, while each CTA has a tile of outputs
  const int64_t out_tiles = (N + (yb ? 127 : 63)) / (yb ? 128 : 64);
  g.shares = int(std::max<int64_t>(1, std::min(clusters_at_once(cl) / tiles, out_tiles / cl)));
  // A tile with several runs takes a product of each for every output tile: idle SMs help with such tiles.
  g.tiles = int(tiles);
  if (g.shares == 1 && tiles <= kMostHelped && out_tiles >= 2 * cl)
    g.helpers = int(std::min<int64_t>(std::max<int64_t>(clusters_at_once(cl) - tiles, 0), tiles));
  if (yb) return tma ? launch_tiles<true, true>(cl, maps, g, s) : launch_tiles<true, false>(cl, maps, g, s);
  return tma ? launch_tiles<false, true>(cl, maps, g, s) : launch_tiles<false, false>(cl, maps, g, s);
}

}  // namespace bl
