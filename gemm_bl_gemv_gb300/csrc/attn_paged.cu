// Attention of new tokens over a paged key-value cache (bl_attn_paged):
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j - max),
// j over the tokens of the request's pages that the new token sees.
//
// A unit is a request's key-value head with up to 16 rows, a row being one
// (new token, query head of the group).  A unit's visible cache is cut into tiles
// of TT tokens, and all tiles of all units, one after the other, are dealt out in
// equal contiguous stretches to the warps of the grid, whatever the lengths are:
// the prefix sums over the requests are formed by every CTA.  A warp is on its own:
// it fetches its tiles by asynchronous copies into its own ring of shared memory,
// several tiles ahead and across units, and keeps the running maximum, sum and
// weighted sum of a unit's rows in registers.  A unit inside one warp's stretch is
// written out at once.  The parts of a unit that is cut by stretches are joined by
// the CTA, where the warps' rings have room for them by then, and those of a unit
// that is cut between CTAs by a second kernel, from the workspace.
//
// The products run on mma.sync m16n8k16 (bf16, fp32 sums): up to 16 rows of queries
// against the tile.  They are bound by the cache's bytes: at the measured copy rate an
// SM receives 12 values of k and v per clock, 190 multiply-adds with 16 rows, of the
// 1017 that mma.sync does.  What bounds the kernel is the issue of the copies (16 bytes
// a lane, some 55 clocks for 32 lanes) and of the weights, and, in short calls, the 6 us
// before the first tile arrives: 64 requests of up to 8192 tokens (40 heads of queries,
// 8 of keys, D 128) 194 us, 5.6 TB/s; 256 of up to 600 73 us; one of 4096 15 us.  12 warps
// with two stages each: with 8 and three, 31.5 us instead of 28.3 for 256 requests of up to
// 100 tokens and 93 instead of 86 for D 80; with 6 and four 40 and 117 (all with weights of
// 16 bits).
// The tensor core cuts its sums off instead of rounding them, so a tile's weighted
// sum starts from zero and is added to the running one in fp32.  The weights go in
// as three bf16 terms, all their 24 bits, so a bf16 result is the fp32 one rounded
// once; two terms (16 bits) move 2 of 1000 bf16 results by a step, and are 1 to 3 %
// faster (D 80 and 256: a tenth).
#include <cmath>

#include "attn_paged.cuh"

namespace bl {
namespace {

using namespace attn;

constexpr int kMostWarps = 12;  // of a CTA

// A warp's part of a unit that is cut by stretches.
struct Part {
  bool present, ends;  // ends: the unit's last tile is in it
  Unit unit;
  int64_t last;        // the unit's last tile
  const float2* stat;  // by row: maximum and sum
  const float* acc;    // [row][D] weighted sums
};

template <int DP_>
struct Shape {
  static constexpr int DP = DP_;
  static constexpr int ROWS = 16;
  static constexpr int TT = DP == 64 ? 32 : 16;        // tokens of a tile
  static constexpr int WARPS = DP == 256 ? 4 : 12;
  static constexpr int STAGES = WARPS == 12 ? 2 : 3;
  static constexpr int CHUNKS = DP / 8;                // 16-byte chunks of a row
  static constexpr int TILE = TT * DP * 2;             // bytes of a tile of k
  static constexpr int SMEM = WARPS * STAGES * 2 * TILE;
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <class S, bool F32>
__global__ void __launch_bounds__(S::WARPS * 32, 1) attn_paged_kernel(const Args a) {
  constexpr int TT = S::TT, NT = TT / 8, KS = S::DP / 16;
  constexpr int kThreads = S::WARPS * 32;
  constexpr uint32_t kAll = TT == 32 ? 0xffffffffu : (1u << TT) - 1;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int64_t before[kThreads + 1];
  __shared__ int64_t warp_total[S::WARPS];
  __shared__ uint32_t real[S::WARPS][S::STAGES];  // tokens of a stage that are there
  // of every warp: its part of a unit begun before its stretch, and of one that goes on behind it
  __shared__ Part parts[S::WARPS][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  pdl_wait();

  // tiles before every share of the requests
  const int64_t share = quotient(a.R + kThreads - 1, kThreads);
  {
    int64_t mine = 0;
    for (int64_t r = tid * share; r < min(a.R, (tid + 1) * share); ++r) {
      const Request q = request_of<S>(a, r);
      mine += int64_t(a.Hk) * q.blocks * q.tiles;
      bad |= q.bad;
    }
    int64_t through = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t w = __shfl_up_sync(0xffffffffu, through, o);
      if (lane >= o) through += w;
    }
    if (lane == 31) warp_total[warp] = through;
    __syncthreads();
    int64_t sum = 0;
    for (int i = 0; i < warp; ++i) sum += warp_total[i];
    before[tid + 1] = sum + through;
    if (tid == 0) before[0] = 0;
    __syncthreads();
  }
  const int64_t all = before[kThreads];
  // equal stretches for the CTAs, and for the warps of a CTA
  const int64_t quota = max(int64_t(1), quotient(all + gridDim.x - 1, gridDim.x));
  const int64_t end = min(all, (blockIdx.x + 1) * quota);
  const int64_t each = (quota + S::WARPS - 1) / S::WARPS;
  const int64_t t0 = blockIdx.x * quota + warp * each;
  const int count = int(max(int64_t(0), min(each, end - t0)));
  if (lane < 2) parts[warp][lane].present = false;
  __syncwarp();

  if (count > 0) {
    Place<S> at;
    at.find(a, before, kThreads, share, t0);
    uint8_t* mine = ring + warp * (S::STAGES * 2 * S::TILE);

    // The page of this lane's token of a tile, -1: none.
    auto page_of = [&](const Place<S>& p) {
      const int j = p.token() + lane;
      if (lane >= TT || j >= p.q.length || (a.window > 0 && j < p.q.low && j >= a.sinks)) return -1;
      const int entry = a.table[p.r * a.W + a.by_page.quotient(j)];
      if (entry < 0 || entry >= a.pages) {
        bad = true;
        return -1;
      }
      return entry;
    };
    // Starts the copies of a tile.  Lane l copies chunk l % CHUNKS of every kRows-th row, from row l / CHUNKS on.
    constexpr int kRows = 32 / S::CHUNKS;
    const int chunk = lane % S::CHUNKS, sub = lane / S::CHUNKS;
    const bool inside = chunk * 8 < a.D;
    const uint32_t lane_to = sub * (S::DP * 2) + ((chunk ^ sub) * 16);  // of row i + sub: xor of the row's low bits
    auto fetch = [&](const Place<S>& p, int entry, int stage) {
      const unsigned there = __ballot_sync(0xffffffffu, entry >= 0);
      if (lane == 0) real[warp][stage] = there;
      const int j0 = p.token();
      const uint32_t k = smem_addr(mine + stage * 2 * S::TILE) + lane_to;
      if (a.tiled) {
        const int one = __shfl_sync(0xffffffffu, entry, __ffs(there) - 1);
        const int64_t at = ((int64_t(max(one, 0)) * a.Hk + p.head()) * a.page + j0 - a.by_page.quotient(j0) * a.page + sub) * a.D + (inside ? chunk * 8 : 0);
        const uint16_t *kf = a.k + at, *vf = a.v + at;
        if (there == kAll) {
#pragma unroll
          for (int i = 0; i < TT; i += kRows) {
            const uint32_t to = (k ^ ((i & 7) * 16)) + i * (S::DP * 2);
            copy16(to, kf + uint32_t(i * a.D), inside);
            copy16(to + S::TILE, vf + uint32_t(i * a.D), inside);
          }
        } else {
#pragma unroll
          for (int i = 0; i < TT; i += kRows) {
            const uint32_t to = (k ^ ((i & 7) * 16)) + i * (S::DP * 2);
            const bool ok = (there >> (i + sub) & 1) && inside;
            copy16(to, kf + (ok ? uint32_t(i * a.D) : 0), ok);
            copy16(to + S::TILE, vf + (ok ? uint32_t(i * a.D) : 0), ok);
          }
        }
      } else {
        const int j = j0 + lane;
        const int64_t base = entry < 0 ? 0 : ((int64_t(entry) * a.Hk + p.head()) * a.page + j - a.by_page.quotient(j) * a.page) * a.D;
#pragma unroll
        for (int i = 0; i < TT; i += kRows) {
          const int64_t from = __shfl_sync(0xffffffffu, base, i + sub) + chunk * 8;
          const bool ok = (there >> (i + sub) & 1) && inside;
          const uint32_t to = (k ^ ((i & 7) * 16)) + i * (S::DP * 2);
          copy16(to, a.k + (ok ? from : 0), ok);
          copy16(to + S::TILE, a.v + (ok ? from : 0), ok);
        }
      }
    };

    // The queries of a unit that begins with the tile to come are asked into L2, a lane per 128 bytes (2.4 us of
    // 64 requests of up to 2000 tokens).
    auto ask_queries = [&](const Place<S>& p) {
      const int row0 = p.row0(), n = min(S::ROWS, int(min(int64_t(p.q.n) * a.G - row0, int64_t(S::ROWS))));
      const int lines = (a.D * 2 + 127) / 128;
      for (int i = lane; i < n * lines; i += 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + row_at(a, {p.q.first, p.head(), row0, n}, i / lines) + min(i % lines * 64, a.D - 8)));
    };
    Place<S> ahead = at;
    ask_queries(ahead);
    int fetched = 0;
    int entry = page_of(ahead);
    auto fetch_next = [&]() {
      if (fetched < count) {
        fetch(ahead, entry, fetched % S::STAGES);
        ++fetched;
        if (fetched < count) {
          ahead.next(a);
          entry = page_of(ahead);
          if (ahead.tile == 0) ask_queries(ahead);
        }
      }
      copies_commit();
    };
#pragma unroll 1
    for (int i = 0; i + 1 < S::STAGES; ++i) fetch_next();

    const int g = lane / 4, c2 = lane % 4 * 2;  // this lane's row (and row + 8) and columns of an accumulator
    uint32_t qf[KS][4];
    float acc[2 * KS][4], top[2], sum[2];
    int mine_at[2];  // a row's position
    int head = 0, row0 = 0, nrows = 0;
    bool begun = false, fresh = true;

#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      if (fresh) {  // a unit begins (or this stretch does)
        fresh = false;
        begun = at.tile == 0;
        head = at.head();
        row0 = at.row0();
        nrows = min(S::ROWS, int(min(int64_t(at.q.n) * a.G - row0, int64_t(S::ROWS))));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int row = g + s * 8;
          const uint16_t* q = a.q + row_at(a, {at.q.first, head, row0, nrows}, row);
          mine_at[s] = at.q.length - at.q.n + a.by_group.quotient(row0 + row);
          top[s] = -INFINITY;
          sum[s] = 0.f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const int d = ks * 16 + c2;
            qf[ks][s] = row < nrows && d < a.D && !a.zero ? *reinterpret_cast<const uint32_t*>(q + d) ^ a.sign : 0;
            qf[ks][s + 2] = row < nrows && d + 8 < a.D && !a.zero ? *reinterpret_cast<const uint32_t*>(q + d + 8) ^ a.sign : 0;
          }
        }
#pragma unroll
        for (int nt = 0; nt < 2 * KS; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
      }
      fetch_next();
      copies_wait<S::STAGES - 1>();
      __syncwarp();
      const int stage = i % S::STAGES;
      const uint32_t k = smem_addr(mine + stage * 2 * S::TILE), v = k + S::TILE;
      const int j0 = at.token();

      // scores
      float z[NT][4];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int p = 0; p < NT / 2; ++p) {
          const int row = p * 16 + (lane / 16) * 8 + (lane & 7), chunk = ks * 2 + (lane / 8 & 1);
          uint32_t b[4];
          ldmatrix4(b, k + row * (S::DP * 2) + ((chunk ^ (row & 7)) * 16));
          if (ks == 0) {
            mma_first(z[2 * p], qf[ks], b[0], b[1]);
            mma_first(z[2 * p + 1], qf[ks], b[2], b[3]);
          } else {
            mma(z[2 * p], qf[ks], b[0], b[1]);
            mma(z[2 * p + 1], qf[ks], b[2], b[3]);
          }
        }
      // Every row sees the whole tile, unless it reaches past the first new token, lies at the window's edge or has
      // tokens that are not there.
      const uint32_t there = real[warp][stage];
      const bool whole = there == kAll && j0 + TT - 1 <= at.q.length - at.q.n &&
                         (a.window <= 0 || j0 + TT <= a.sinks || j0 > int64_t(at.q.length) - 1 - a.window);
      auto sees = [&](int at_row, int j) {
        return (there >> (j - j0) & 1) && j <= at_row && (a.window <= 0 || j > at_row - a.window || j < a.sinks);
      };
      if (!whole) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!sees(mine_at[e / 2], j0 + nt * 8 + c2 + (e & 1))) z[nt][e] = -INFINITY;
      }
      // weights
      float keep[2];  // what the sums so far are multiplied by
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float m = top[s];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) m = fmaxf(m, fmaxf(z[nt][2 * s], z[nt][2 * s + 1]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const float base = m == -INFINITY ? 0.f : m;  // nothing seen yet: all weights are 0
        const float shift = base * a.scale;
        keep[s] = exp2_fast((top[s] - base) * a.scale);
        top[s] = m;
        float add = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 2 * s; e < 2 * s + 2; ++e) {
            z[nt][e] = exp2_fast(__fmaf_rn(z[nt][e], a.scale, -shift));
            add += z[nt][e];
          }
        sum[s] = __fmaf_rn(sum[s], keep[s], add);
      }
      // A value that some rows do not see must not reach them, and 0 times an infinity or NaN would: such tiles
      // are looked through, and added up value by value where there is one.
      bool apart = false;
      if (!whole) {
        uint32_t odd = 0;
#pragma unroll 4
        for (int i4 = lane; i4 < TT * S::CHUNKS; i4 += 32) {
          uint4 w;
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(v + i4 * 16) : "memory");
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) odd |= (u[j] & 0x7f80u) == 0x7f80u || (u[j] & 0x7f800000u) == 0x7f800000u;
        }
        apart = __any_sync(0xffffffffu, odd != 0);
      }
      if (!apart) {
        uint32_t w[TT / 16][TERMS][4];
#pragma unroll
        for (int p = 0; p < TT / 16; ++p)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo = z[2 * p + e / 2][2 * (e & 1)], hi = z[2 * p + e / 2][2 * (e & 1) + 1];
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
              const uint32_t u = bf16x2_rn(lo, hi);
              w[p][t][e] = u;
              lo -= __uint_as_float(u << 16);
              hi -= __uint_as_float(u & 0xffff0000u);
            }
          }
#pragma unroll
        for (int np = 0; np < KS; ++np) {
          uint32_t b[TT / 16][4];
#pragma unroll
          for (int p = 0; p < TT / 16; ++p) {
            const int row = p * 16 + (lane & 15), chunk = np * 2 + lane / 16;
            ldmatrix4_trans(b[p], v + row * (S::DP * 2) + ((chunk ^ (row & 7)) * 16));
          }
          float o0[4], o1[4];
#pragma unroll
          for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
            for (int p = 0; p < TT / 16; ++p) {
              if (t == TERMS - 1 && p == 0) {
                mma_first(o0, w[p][t], b[p][0], b[p][1]);
                mma_first(o1, w[p][t], b[p][2], b[p][3]);
              } else {
                mma(o0, w[p][t], b[p][0], b[p][1]);
                mma(o1, w[p][t], b[p][2], b[p][3]);
              }
            }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[2 * np][e] = __fmaf_rn(acc[2 * np][e], keep[e / 2], o0[e]);
            acc[2 * np + 1][e] = __fmaf_rn(acc[2 * np + 1][e], keep[e / 2], o1[e]);
          }
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < 2 * KS; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][e] *= keep[e / 2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll 1
          for (int jj = 0; jj < 8; ++jj) {
            const int row = nt * 8 + jj, from = g * 4 + jj / 2;
            float wr[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const float even = __shfl_sync(0xffffffffu, z[nt][2 * s], from);
              const float uneven = __shfl_sync(0xffffffffu, z[nt][2 * s + 1], from);
              wr[s] = jj & 1 ? uneven : even;
            }
            const bool see0 = sees(mine_at[0], j0 + row), see1 = sees(mine_at[1], j0 + row);
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n) {
              uint32_t u;
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(v + row * (S::DP * 2) + ((n ^ (row & 7)) * 16) + c2 * 2) : "memory");
              const float v0 = __uint_as_float(u << 16), v1 = __uint_as_float(u & 0xffff0000u);
              if (see0) {
                acc[n][0] = __fmaf_rn(wr[0], v0, acc[n][0]);
                acc[n][1] = __fmaf_rn(wr[0], v1, acc[n][1]);
              }
              if (see1) {
                acc[n][2] = __fmaf_rn(wr[1], v0, acc[n][2]);
                acc[n][3] = __fmaf_rn(wr[1], v1, acc[n][3]);
              }
            }
          }
      }
      __syncwarp();  // the stage has been read

      const bool ends = at.tile + 1 == at.q.tiles;
      if (ends || i + 1 == count) {
        const bool out = begun && ends;
        // the ring is free at the stretch's end; a part that ends before it waits in the workspace
        const bool final = i + 1 == count;
        if (final) {
          copies_wait<0>();
          __syncwarp();
        }
        const int64_t slot = 2 * int64_t(gridDim.x) + blockIdx.x * S::WARPS + warp;
        float2* stat = final ? reinterpret_cast<float2*>(mine) : a.stat + slot * a.rows;
        float* sums = final ? reinterpret_cast<float*>(mine + S::ROWS * sizeof(float2)) : a.acc + slot * a.rows * a.D;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float l = sum[s];
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          const int row = g + s * 8;
          if (row >= nrows) continue;
          if (out) {
            const int64_t to = row_at(a, {at.q.first, head, row0, nrows}, row);
            const float inv = top[s] == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n)
              if (n * 8 < a.D) {
                const float x = acc[n][2 * s] * inv, y = acc[n][2 * s + 1] * inv;
                if (F32)
                  *reinterpret_cast<float2*>(static_cast<float*>(a.out) + to + n * 8 + c2) = make_float2(x, y);
                else
                  *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to + n * 8 + c2) = bf16x2_rn(x, y);
              }
          } else {
            if (lane % 4 == 0) stat[row] = make_float2(top[s], l);
            float* to = sums + row * a.D;
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n)
              if (n * 8 < a.D)
                *reinterpret_cast<float2*>(to + n * 8 + c2) = make_float2(acc[n][2 * s], acc[n][2 * s + 1]);
          }
        }
        if (!out && lane == 0)
          parts[warp][begun] = {true, ends, {at.q.first, head, row0, nrows}, t0 + i + (at.q.tiles - 1 - at.tile), stat, sums};
        fresh = true;
      }
      if (i + 1 < count) at.next(a);
    }
  }
  // The units that are cut: each begins with a part that goes on (or, the first, with what an earlier CTA began) and
  // runs through the next warps' parts.  A warp joins every WARPS-th row of all of them.
  const bool any_bad = __syncthreads_or(bad);
  if (any_bad && tid == 0) atomicOr(a.err, BL_DEVERR_RANGE);
  const Part& of_lane = parts[min(lane, S::WARPS - 1)][0];
  const bool mine = lane < S::WARPS;
  const unsigned goes_on = __ballot_sync(0xffffffffu, mine && of_lane.present && !of_lane.ends);  // through the whole stretch
  const unsigned ended = __ballot_sync(0xffffffffu, mine && of_lane.present && of_lane.ends);
  const unsigned begins = __ballot_sync(0xffffffffu, mine && parts[min(lane, S::WARPS - 1)][1].present);
  if (tid == 0) {
    Header header = {};
    const Part& last = parts[31 - __clz(begins | 1)][1];  // the unit that goes on behind the CTA, if one does
    if (begins && last.last >= end) {
      header.unit = last.unit;
      header.present = 1;
      header.follow = int(quotient(last.last, quota) - blockIdx.x);
    }
    a.header[blockIdx.x] = header;
  }
  int task = warp;
  // a bit per unit: 0 for one that was begun before this CTA, w + 1 for one that begins in warp w's stretch
  for (unsigned todo = begins << 1 | ((goes_on | ended) & 1); todo; todo &= todo - 1) {
    const int w0 = __ffs(todo) - 2, from = max(w0, 0);
    const Part& first = w0 < 0 ? parts[0][0] : parts[w0][1];
    int n = 1;
    if (w0 >= 0 || !(ended & 1)) {  // the next warps' parts, up to one that ends
      const unsigned rest = ~goes_on >> (from + 1);  // its lowest bit: the first that does not go on
      const int through = __ffs(rest) - 1;
      n += through + (ended >> (from + 1 + through) & 1);
    }
    auto part = [&](int p) -> const Part& { return p == 0 ? first : parts[from + p][0]; };
    for (; task < first.unit.n; task += S::WARPS) {
      const int row = task;
      join_row(a, n, [&](int p) { return part(p).stat[row]; }, [&](int p) { return part(p).acc + row * a.D; },
               [&](float l, float top, const float4(&o)[2]) {
                 if (w0 >= 0 && first.last < end) {
                   store_row<F32>(a, row_at(a, first.unit, row), l, top, o);
                 } else {
                   const int64_t to = (2 * int64_t(blockIdx.x) + (w0 >= 0)) * a.rows + row;
                   if (lane == 0) a.stat[to] = make_float2(top, l);
#pragma unroll
                   for (int i = 0; i < 2; ++i)
                     if (lane + 32 * i < a.D / 4) reinterpret_cast<float4*>(a.acc + to * a.D)[lane + 32 * i] = o[i];
                 }
               });
    }
    task -= first.unit.n;
  }
  pdl_launch_dependents();
}

// Joins the parts of the units that are cut between CTAs: a CTA looks at one header, a warp takes rows.
template <bool F32>
__global__ void __launch_bounds__(128) attn_join_kernel(const Args a) {
  pdl_wait();
  const Header hd = a.header[blockIdx.x];
  if (hd.present) {
    // part p: what the first CTA left of a unit that begins in it, then what the next ones have of a unit begun before
    auto part = [&](int p) { return 2 * int64_t(blockIdx.x + p) + (p == 0); };
    for (int row = blockIdx.y * 4 + (threadIdx.x >> 5); row < hd.unit.n; row += gridDim.y * 4)
      join_row(a, 1 + hd.follow, [&](int p) { return a.stat[part(p) * a.rows + row]; },
               [&](int p) { return a.acc + (part(p) * a.rows + row) * a.D; },
               [&](float l, float top, const float4(&o)[2]) { store_row<F32>(a, row_at(a, hd.unit, row), l, top, o); });
  }
  pdl_launch_dependents();
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Rows that a part keeps at most.
int part_rows(int64_t M, int H, int Hk, int D) {
  return int(std::min<int64_t>(D <= 128 ? 32 : 16, M * (H / Hk)));
}

template <class S, bool F32>
cudaError_t launch_as(const Args& given, cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = raise_smem_cap(attn_paged_kernel<S, F32>, dev, S::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sm_count(), kMostCtas);
  Args a = given;
  a.tiled = a.page % S::TT == 0;
  e = launch(attn_paged_kernel<S, F32>, dim3(grid), dim3(S::WARPS * 32), S::SMEM, s, overlap_enabled(), a);
  if (e != cudaSuccess) return e;
  // The join waits for the whole first kernel, so the two may overlap in either setting.
  return launch(attn_join_kernel<F32>, dim3(grid, S::ROWS / 4), dim3(128), 0, s, true, a);
}

template <bool F32>
cudaError_t launch_for(const Args& a, cudaStream_t s) {
  // Units of 32 rows with tiles of 128 tokens by TMA on tcgen05, or of 16 rows with tiles of 16 (32) by each warp on mma.sync.
  // The former takes 1.3 us a tile, however many rows there are, with 1 to 4 us for a unit; the latter less for a short unit,
  // and twice as much for more than 16 rows.  So tcgen05 has requests with ten rows of a key-value head and more, and D 104 to
  // 128 where the tables have room for long requests (the lengths are known on the device only).  Measured, mma.sync / tcgen05,
  // us, requests x (evenly spread) lengths up to, 20/5 query / key heads, D 128 and pages of 16 unless stated:
  //   rows: 256 x 600: 2 new tokens (8 rows) 83/96, 3: 97/97, 5: 143/97; 64 x 300, 5 new 41/26; 64 x 1000, 32/8, 8 new
  //     108/61; 48 x 20000, 40/8, 5 new, window 4096, fp32 234/139; D 80, 64 x 1000, 5 new 61/42; D 64 37/42.
  //   one token: 64 x 8192, 40/8 194/180, pages of 64 194/173; 3 x 131072 116/112; 1 x 4096 15.2/14.8; 4 x 30000, 8/8 62/61;
  //     and 64 x 2000 49/56; 16 x 1000 17/21; 256 x 600 73/96; 256 x 100 29/44; D 80, 8 x 30000, 40/8 97/93; D 64, 64 x 4000,
  //     16/8 57/111.
  const bool rows = a.M * a.G >= 10 * a.R, room = a.D > 96 && a.W * a.page >= 4096;
  if (a.D > 64 && a.D <= 128 && (rows || room)) {
    const int grid = std::min(sm_count(), kMostCtas);
    const cudaError_t e = launch_tc(a, grid, F32, s);
    if (e == cudaSuccess) return launch(attn_join_kernel<F32>, dim3(grid, 8), dim3(128), 0, s, true, a);
    if (e != cudaErrorNotSupported) return e;  // else: pages that it has no boxes for
  }
  if (a.D <= 64) return launch_as<Shape<64>, F32>(a, s);
  if (a.D <= 128) return launch_as<Shape<128>, F32>(a, s);
  return launch_as<Shape<256>, F32>(a, s);
}

}  // namespace

constexpr size_t kMostParts = size_t(kMostCtas) * (2 + kMostWarps);

size_t attn_paged_workspace(int64_t M, int H, int Hk, int D) {
  const size_t rows = part_rows(M, H, Hk, D);
  return align256(kMostCtas * sizeof(Header)) + align256(kMostParts * rows * sizeof(float2)) + kMostParts * rows * D * sizeof(float);
}

cudaError_t launch_attn_paged(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache, const int32_t* table,
                              const int32_t* length, const int32_t* start, float scale, int64_t window, int64_t sinks,
                              int64_t M, int64_t R, int H, int Hk, int D, int64_t pages, int page, int64_t W, void* out,
                              bl_dtype ot, uint8_t* ws, cudaStream_t s) {
  Args a{q, k_cache, v_cache, table, length, start, out};
  a.err = dev_error_ptr();
  if (!a.err) return cudaErrorUnknown;
  a.M = M, a.R = R, a.pages = pages, a.W = W;
  a.H = H, a.Hk = Hk, a.G = H / Hk, a.D = D, a.page = page, a.rows = part_rows(M, H, Hk, D);
  a.window = std::min(window, int64_t(1) << 31), a.sinks = std::min(sinks, int64_t(1) << 31);  // all tokens: sums of them stay in 64 bits
  // The kernel works with a positive factor, whose largest score is the largest sum: the sign goes to the queries, and
  // with a scale of 0 all of them (times any key) are 0.
  a.scale = scale == 0.f ? 1.f : std::fabs(scale) * 1.4426950408889634f;
  a.sign = scale < 0.f ? 0x80008000u : 0u;
  a.zero = scale == 0.f;
  a.wait_ns = wait_limit_ns();
  a.by_page.set(uint32_t(page));
  a.by_group.set(uint32_t(a.G));
  a.header = reinterpret_cast<Header*>(ws);
  ws += align256(kMostCtas * sizeof(Header));
  a.stat = reinterpret_cast<float2*>(ws);
  ws += align256(kMostParts * a.rows * sizeof(float2));
  a.acc = reinterpret_cast<float*>(ws);
  return ot == BL_F32 ? launch_for<true>(a, s) : launch_for<false>(a, s);
}

}  // namespace bl
