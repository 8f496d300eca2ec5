// Attention of new tokens over a paged key-value cache (bl_attn_paged):
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j - max),
// j over the tokens of the request's pages that the new token sees.
//
// A unit is a request's key-value head with up to 16 MT rows, a row being one
// (new token, query head of the group).  A unit's visible cache is cut into tiles
// of TT tokens, and all tiles of all units, one after the other, are dealt out in
// equal contiguous stretches to the warps of the grid, whatever the lengths are:
// the prefix sums over the requests are formed by every CTA.  A warp is on its own:
// it fetches its tiles by asynchronous copies into its own ring of shared memory,
// several tiles ahead and across units, and keeps the running maximum, sum and
// weighted sum of a unit's rows in registers.  A unit inside one warp's stretch is
// written out at once; of a unit cut by stretches each warp leaves its part in the
// workspace, and a second kernel joins the parts.
//
// The products run on mma.sync m16n8k16 (bf16, fp32 sums): up to 16 rows of queries
// against the tile.  They are bound by the cache's bytes: at the measured copy rate an
// SM receives 12 values of k and v per clock, 190 multiply-adds with 16 rows, of the
// 1017 that mma.sync does (tcgen05's tiles of 64 to 128 rows would be 4/5 empty).
// The tensor core cuts its sums off instead of rounding them, so a tile's weighted
// sum starts from zero and is added to the running one in fp32.  The weights go in
// as two bf16 terms (16 bits) for bf16 results, three (24 bits) for fp32 ones.
#include "bl_device.cuh"
#include "bl_internal.h"
#include "paged.cuh"

namespace bl {
namespace {

constexpr int kMostCtas = 160;  // of the first kernel, for the size of the workspace
constexpr int kMostWarps = 8;   // of a CTA

// What a warp leaves of the unit that goes on in the next warp's stretch.
struct __align__(16) Header {
  int present;
  int token;    // first new token of the request
  int head;     // key-value head
  int row0, n;  // the unit's rows: n from row0 on
  int follow;   // warps after this one that have a part
  int pad[2];
};

struct Args {
  const uint16_t *q, *k, *v;
  const int32_t *table, *length, *start;
  void* out;
  Header* header;
  float2* stat;  // (max, sum) of each row of each part
  float* acc;    // weighted sums
  int64_t M, R, pages, W;
  int H, Hk, G, D, page, rows;  // rows: kept of a part
  int64_t window, sinks;
  float scale;  // times log2(e)
  unsigned int* err;
};

template <int DP_, int MT_>
struct Shape {
  static constexpr int DP = DP_, MT = MT_;
  static constexpr int ROWS = 16 * MT;
  static constexpr int TT = DP == 64 ? 32 : 16;        // tokens of a tile
  static constexpr int WARPS = DP == 256 ? 4 : 8;
  static constexpr int STAGES = 3;
  static constexpr int CHUNKS = DP / 8;                // 16-byte chunks of a row
  static constexpr int TILE = TT * DP * 2;             // bytes of a tile of k
  static constexpr int SMEM = WARPS * STAGES * 2 * TILE;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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
// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __forceinline__ Request request_of(const Args& a, int64_t r) {
  Request q;
  const Rows rows = rows_of(a.start, r, a.M);
  q.first = rows.first;
  q.n = rows.n;
  const int64_t most = min(a.W * a.page, int64_t(INT32_MAX));
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

template <class S, bool F32>
__global__ void __launch_bounds__(S::WARPS * 32, 1) attn_paged_kernel(const Args a) {
  constexpr int TT = S::TT, NT = TT / 8, KS = S::DP / 16, MT = S::MT, TERMS = F32 ? 3 : 2;
  constexpr int kThreads = S::WARPS * 32;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int64_t before[kThreads + 1];
  __shared__ int64_t warp_total[S::WARPS];
  __shared__ uint32_t real[S::WARPS][S::STAGES];  // tokens of a stage that are there
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  pdl_wait();

  // tiles before every share of the requests
  const int64_t share = (a.R + kThreads - 1) / kThreads;
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
  const int64_t warps = int64_t(gridDim.x) * S::WARPS;
  const int64_t quota = max(int64_t(1), (all + warps - 1) / warps);
  // neighbouring stretches lie on different SMs, so that few tiles spread over all of them
  const int64_t me = int64_t(warp) * gridDim.x + blockIdx.x;
  const int64_t t0 = me * quota;
  const int count = int(max(int64_t(0), min(quota, all - t0)));
  Header header = {};

  if (count > 0) {
    // the first tile
    Place<S> at;
    {
      int lo = 0, hi = kThreads;  // before[lo] <= t0 < before[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (before[mid] <= t0)
          lo = mid;
        else
          hi = mid;
      }
      int64_t rest = t0 - before[lo];
      for (at.r = lo * share;; ++at.r) {
        at.q = request_of<S>(a, at.r);
        const int64_t tiles = int64_t(a.Hk) * at.q.blocks * at.q.tiles;
        if (rest < tiles) break;
        rest -= tiles;
      }
      at.unit = int(rest / at.q.tiles);
      at.tile = int(rest % at.q.tiles);
    }
    uint8_t* mine = ring + warp * (S::STAGES * 2 * S::TILE);

    // The row of the cache (page * page size + offset) of this lane's token of a tile, -1: none.
    auto row_of = [&](const Place<S>& p) {
      const int j = p.token() + lane;
      if (lane >= TT || j >= p.q.length || (a.window > 0 && j < p.q.low && j >= a.sinks)) return -1;
      const int entry = a.table[p.r * a.W + j / a.page];
      if (entry < 0 || entry >= a.pages) {
        bad = true;
        return -1;
      }
      return entry;
    };
    // Starts the copies of a tile; `entry`: this lane's token's page.
    auto fetch = [&](const Place<S>& p, int entry, int stage) {
      const int j = p.token() + lane;
      const unsigned there = __ballot_sync(0xffffffffu, entry >= 0);
      if (lane == 0) real[warp][stage] = there;
      const int64_t base = entry < 0 ? 0 : ((int64_t(entry) * a.Hk + p.head()) * a.page + j % a.page) * a.D;
      const uint32_t k = smem_addr(mine + stage * 2 * S::TILE), v = k + S::TILE;
      constexpr int kRows = 32 / S::CHUNKS;  // rows that the warp copies at a time
      const int chunk = lane % S::CHUNKS, sub = lane / S::CHUNKS;
#pragma unroll
      for (int i = 0; i < TT; i += kRows) {
        const int row = i + sub;
        const int64_t from = __shfl_sync(0xffffffffu, base, row) + chunk * 8;
        const bool ok = (there >> row & 1) && chunk * 8 < a.D;
        const uint32_t to = row * (S::DP * 2) + ((chunk ^ (row & 7)) * 16);
        copy16(k + to, a.k + (ok ? from : 0), ok);
        copy16(v + to, a.v + (ok ? from : 0), ok);
      }
    };

    Place<S> ahead = at;
    int fetched = 0;
    int entry = row_of(ahead);
    auto fetch_next = [&]() {
      if (fetched < count) {
        fetch(ahead, entry, fetched % S::STAGES);
        ++fetched;
        if (fetched < count) {
          ahead.next(a);
          entry = row_of(ahead);
        }
      }
      copies_commit();
    };
#pragma unroll 1
    for (int i = 0; i + 1 < S::STAGES; ++i) fetch_next();

    const int g = lane / 4, c2 = lane % 4 * 2;  // this lane's row (and row + 8) and columns of an accumulator
    uint32_t qf[MT][KS][4];
    float acc[MT][2 * KS][4], top[MT][2], sum[MT][2];
    int mine_at[MT][2];  // a row's position
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
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int row = mt * 16 + g + s * 8;
            const int t = (row0 + row) / a.G, h = (row0 + row) % a.G;
            const uint16_t* q = a.q + ((int64_t(at.q.first) + t) * a.H + head * a.G + h) * a.D;
            mine_at[mt][s] = at.q.length - at.q.n + t;
            top[mt][s] = -INFINITY;
            sum[mt][s] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const int d = ks * 16 + c2;
              qf[mt][ks][s] = row < nrows && d < a.D ? *reinterpret_cast<const uint32_t*>(q + d) : 0;
              qf[mt][ks][s + 2] = row < nrows && d + 8 < a.D ? *reinterpret_cast<const uint32_t*>(q + d + 8) : 0;
            }
          }
#pragma unroll
          for (int nt = 0; nt < 2 * KS; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
        }
      }
      fetch_next();
      copies_wait<S::STAGES - 1>();
      __syncwarp();
      const int stage = i % S::STAGES;
      const uint32_t k = smem_addr(mine + stage * 2 * S::TILE), v = k + S::TILE;
      const int j0 = at.token();

      // scores
      float z[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[mt][nt][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int p = 0; p < NT / 2; ++p) {
          const int row = p * 16 + (lane / 16) * 8 + (lane & 7), chunk = ks * 2 + (lane / 8 & 1);
          uint32_t b[4];
          ldmatrix4(b, k + row * (S::DP * 2) + ((chunk ^ (row & 7)) * 16));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma(z[mt][2 * p], qf[mt][ks], b[0], b[1]);
            mma(z[mt][2 * p + 1], qf[mt][ks], b[2], b[3]);
          }
        }
      // Every row sees the whole tile, unless it reaches past the first new token, lies at the window's edge or has
      // tokens that are not there.
      const uint32_t there = real[warp][stage];
      constexpr uint32_t kAll = TT == 32 ? 0xffffffffu : (1u << TT) - 1;
      const bool whole = there == kAll && j0 + TT - 1 <= at.q.length - at.q.n &&
                         (a.window <= 0 || j0 + TT <= a.sinks || j0 > int64_t(at.q.length) - 1 - a.window);
      auto sees = [&](int at_row, int j) {
        return (there >> (j - j0) & 1) && j <= at_row && (a.window <= 0 || j > at_row - a.window || j < a.sinks);
      };
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            z[mt][nt][e] *= a.scale;
            if (!whole && !sees(mine_at[mt][e / 2], j0 + nt * 8 + c2 + (e & 1))) z[mt][nt][e] = -INFINITY;
          }
      // weights
      float keep[MT][2];  // what the sums so far are multiplied by
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float m = top[mt][s];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) m = fmaxf(m, fmaxf(z[mt][nt][2 * s], z[mt][nt][2 * s + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const float base = m == -INFINITY ? 0.f : m;  // nothing seen yet: all weights are 0
          keep[mt][s] = exp2_fast(top[mt][s] - base);
          top[mt][s] = m;
          float add = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 2 * s; e < 2 * s + 2; ++e) {
              z[mt][nt][e] = exp2_fast(z[mt][nt][e] - base);
              add += z[mt][nt][e];
            }
          sum[mt][s] = __fmaf_rn(sum[mt][s], keep[mt][s], add);
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
        uint32_t w[MT][TT / 16][TERMS][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int p = 0; p < TT / 16; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo = z[mt][2 * p + e / 2][2 * (e & 1)], hi = z[mt][2 * p + e / 2][2 * (e & 1) + 1];
#pragma unroll
              for (int t = 0; t < TERMS; ++t) {
                const uint32_t u = bf16x2_rn(lo, hi);
                w[mt][p][t][e] = u;
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
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float o0[4] = {0.f, 0.f, 0.f, 0.f}, o1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
              for (int p = 0; p < TT / 16; ++p) {
                mma(o0, w[mt][p][t], b[p][0], b[p][1]);
                mma(o1, w[mt][p][t], b[p][2], b[p][3]);
              }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[mt][2 * np][e] = __fmaf_rn(acc[mt][2 * np][e], keep[mt][e / 2], o0[e]);
              acc[mt][2 * np + 1][e] = __fmaf_rn(acc[mt][2 * np + 1][e], keep[mt][e / 2], o1[e]);
            }
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int nt = 0; nt < 2 * KS; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][nt][e] *= keep[mt][e / 2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll 1
            for (int jj = 0; jj < 8; ++jj) {
              const int row = nt * 8 + jj, from = g * 4 + jj / 2;
              float wr[2];
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const float even = __shfl_sync(0xffffffffu, z[mt][nt][2 * s], from);
                const float uneven = __shfl_sync(0xffffffffu, z[mt][nt][2 * s + 1], from);
                wr[s] = jj & 1 ? uneven : even;
              }
              const bool see0 = sees(mine_at[mt][0], j0 + row), see1 = sees(mine_at[mt][1], j0 + row);
#pragma unroll
              for (int n = 0; n < 2 * KS; ++n) {
                uint32_t u;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(v + row * (S::DP * 2) + ((n ^ (row & 7)) * 16) + c2 * 2) : "memory");
                const float v0 = __uint_as_float(u << 16), v1 = __uint_as_float(u & 0xffff0000u);
                if (see0) {
                  acc[mt][n][0] = __fmaf_rn(wr[0], v0, acc[mt][n][0]);
                  acc[mt][n][1] = __fmaf_rn(wr[0], v1, acc[mt][n][1]);
                }
                if (see1) {
                  acc[mt][n][2] = __fmaf_rn(wr[1], v0, acc[mt][n][2]);
                  acc[mt][n][3] = __fmaf_rn(wr[1], v1, acc[mt][n][3]);
                }
              }
            }
        }
      }
      __syncwarp();  // the stage has been read

      const bool ends = at.tile + 1 == at.q.tiles;
      if (ends || i + 1 == count) {
        const bool out = begun && ends;
        const int64_t part = 2 * me + (begun ? 1 : 0);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            float l = sum[mt][s];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int row = mt * 16 + g + s * 8;
            if (row >= nrows) continue;
            if (out) {
              const int t = (row0 + row) / a.G, h = (row0 + row) % a.G;
              const int64_t to = ((int64_t(at.q.first) + t) * a.H + head * a.G + h) * a.D;
              const float inv = top[mt][s] == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
              for (int n = 0; n < 2 * KS; ++n)
                if (n * 8 < a.D) {
                  const float x = acc[mt][n][2 * s] * inv, y = acc[mt][n][2 * s + 1] * inv;
                  if (F32)
                    *reinterpret_cast<float2*>(static_cast<float*>(a.out) + to + n * 8 + c2) = make_float2(x, y);
                  else
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to + n * 8 + c2) = bf16x2_rn(x, y);
                }
            } else {
              if (lane % 4 == 0) a.stat[part * a.rows + row] = make_float2(top[mt][s], l);
              float* to = a.acc + (part * a.rows + row) * a.D;
#pragma unroll
              for (int n = 0; n < 2 * KS; ++n)
                if (n * 8 < a.D)
                  *reinterpret_cast<float2*>(to + n * 8 + c2) = make_float2(acc[mt][n][2 * s], acc[mt][n][2 * s + 1]);
            }
          }
        if (begun && !ends) {
          const int64_t last = t0 + i + (at.q.tiles - 1 - at.tile);  // the unit's last tile
          header = {1, at.q.first, head, row0, nrows, int(last / quota - me), {0, 0}};
        }
        fresh = true;
      }
      if (i + 1 < count) at.next(a);
    }
    copies_wait<0>();
  }
  if (lane == 0) a.header[me] = header;
  if (__syncthreads_or(bad) && tid == 0) atomicOr(a.err, BL_DEVERR_RANGE);
  pdl_launch_dependents();
}

// Joins the parts of the units that were cut: a CTA looks at the headers of 8 warps, a warp takes rows.
template <bool F32>
__global__ void __launch_bounds__(128) attn_join_kernel(const Args a, int64_t warps) {
  const int lane = threadIdx.x & 31;
  const int first_row = blockIdx.y * 4 + (threadIdx.x >> 5), step = gridDim.y * 4;
  pdl_wait();
  for (int64_t w = int64_t(blockIdx.x) * 8; w < min(warps, int64_t(blockIdx.x) * 8 + 8); ++w) {
    const Header hd = a.header[w];
    if (!hd.present) continue;
    const int parts = 1 + hd.follow;
    // part p: what the first warp left of a unit that begins in it, then what the next ones have of a unit begun before
    auto part = [&](int p) { return p == 0 ? 2 * w + 1 : 2 * (w + p); };
    for (int row = first_row; row < hd.n; row += step) {
      float top = -INFINITY;
      for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.stat[part(p) * a.rows + row].x);
      top = warp_max(top);
      const float base = top == -INFINITY ? 0.f : top;
      float l = 0.f;
      float4 o[2] = {};
      for (int p0 = 0; p0 < parts; p0 += 32) {
        float f = 0.f;
        if (p0 + lane < parts) {
          const float2 s = a.stat[part(p0 + lane) * a.rows + row];
          f = exp2_fast(s.x - base);
          l = __fmaf_rn(f, s.y, l);
        }
        const int n = min(32, parts - p0);
#pragma unroll 4
        for (int p = 0; p < n; ++p) {
          const float fp = __shfl_sync(0xffffffffu, f, p);
          const float4* x = reinterpret_cast<const float4*>(a.acc + (part(p0 + p) * a.rows + row) * a.D);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (lane + 32 * i < a.D / 4) {
              const float4 y = x[lane + 32 * i];
              o[i].x = __fmaf_rn(fp, y.x, o[i].x);
              o[i].y = __fmaf_rn(fp, y.y, o[i].y);
              o[i].z = __fmaf_rn(fp, y.z, o[i].z);
              o[i].w = __fmaf_rn(fp, y.w, o[i].w);
            }
        }
      }
      l = warp_sum(l);
      const float inv = top == -INFINITY && l == 0.f ? 0.f : 1.f / l;
      const int t = (hd.row0 + row) / a.G, h = (hd.row0 + row) % a.G;
      const int64_t to = ((int64_t(hd.token) + t) * a.H + hd.head * a.G + h) * a.D;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < a.D / 4) {
          const int64_t d = to + (lane + 32 * i) * 4;
          if (F32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + d) =
                make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + d) =
                make_uint2(bf16x2_rn(o[i].x * inv, o[i].y * inv), bf16x2_rn(o[i].z * inv, o[i].w * inv));
        }
    }
  }
  pdl_launch_dependents();
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Rows that a part keeps at most.
int part_rows(int64_t M, int H, int Hk, int D) {
  return int(std::min<int64_t>(D <= 128 ? 32 : 16, M * (H / Hk)));
}

template <class S, bool F32>
cudaError_t launch_as(const Args& a, cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = raise_smem_cap(attn_paged_kernel<S, F32>, dev, S::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sm_count(), kMostCtas);
  e = launch(attn_paged_kernel<S, F32>, dim3(grid), dim3(S::WARPS * 32), S::SMEM, s, overlap_enabled(), a);
  if (e != cudaSuccess) return e;
  const int64_t warps = int64_t(grid) * S::WARPS;
  // The join waits for the whole first kernel, so the two may overlap in either setting.
  return launch(attn_join_kernel<F32>, dim3(unsigned((warps + 7) / 8), S::ROWS / 4), dim3(128), 0, s, true, a, warps);
}

template <bool F32>
cudaError_t launch_for(const Args& a, cudaStream_t s) {
  // Two blocks of 16 rows share a tile where the requests have, on the average, more than 16 rows.
  const bool two = (a.M + a.R - 1) / a.R * a.G > 16;
  if (a.D <= 64) return two ? launch_as<Shape<64, 2>, F32>(a, s) : launch_as<Shape<64, 1>, F32>(a, s);
  if (a.D <= 128) return two ? launch_as<Shape<128, 2>, F32>(a, s) : launch_as<Shape<128, 1>, F32>(a, s);
  return launch_as<Shape<256, 1>, F32>(a, s);
}

}  // namespace

size_t attn_paged_workspace(int64_t M, int H, int Hk, int D) {
  const size_t warps = size_t(kMostCtas) * kMostWarps, rows = part_rows(M, H, Hk, D);
  return align256(warps * sizeof(Header)) + align256(2 * warps * rows * sizeof(float2)) + 2 * warps * rows * D * sizeof(float);
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
  a.window = window, a.sinks = sinks, a.scale = scale * 1.4426950408889634f;
  const size_t warps = size_t(kMostCtas) * kMostWarps;
  a.header = reinterpret_cast<Header*>(ws);
  ws += align256(warps * sizeof(Header));
  a.stat = reinterpret_cast<float2*>(ws);
  ws += align256(2 * warps * a.rows * sizeof(float2));
  a.acc = reinterpret_cast<float*>(ws);
  return ot == BL_F32 ? launch_for<true>(a, s) : launch_for<false>(a, s);
}

}  // namespace bl
