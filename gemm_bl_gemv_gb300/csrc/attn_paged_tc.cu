// Attention of new tokens over a paged key-value cache (bl_attn_paged) on the 5th-generation tensor cores, for requests
// whose new tokens make many rows of a key-value head (drafts), D <= 128.
//
// Units, tiles and stretches are those of the other kernel (attn_paged.cu), with tiles of 128 tokens, and the CTA as the
// one worker of a stretch.  A unit has up to NR rows, and the products stand on their sides, so that the few rows are the
// short dimension:
//   S^T [128 tokens x NR]  = K [tokens x D] Q^T,           a tile of k as it lies in the cache, K-major
//   O^T [D x TERMS NR]     = V^T [D x tokens] P^T,         a tile of v as it lies in the cache, M-major
// A thread then has a token's scores of half of the rows, or a coordinate's sums of all: nothing is exchanged between
// threads in a tile, unless a row's maximum rises by more than 2^8: weights are beside a maximum that may be that much
// out of date.  A row that has seen nothing yet has one below all scores, so that the first that it sees raises it.  The
// weights' bf16 terms (three, all their 24 bits) are TERMS rows of P each, so one pass over v does for all.  The tensor
// core cuts its sums off instead of rounding them; a tile's sums start from zero and are added to the running ones in
// registers, in fp32.
//
// Warps: 0-7 weights; 8-11 sums; 12 and 13 start the copies of k and v (TMA boxes of a page's rows, zeros for a page that
// is not there); 14 products; 15 looks ahead: the pages of the next tiles' tokens.  k and v of a tile share a ring of
// five half tiles.  A page is 128 tokens or more in steps of 128, or 8, 16, 32 or 64; the other kernel takes others.
//
// Bound: HBM where lengths are long (64 requests of up to 8192 tokens, 40 / 8 heads, one new token: 180 us, 6.1 TB/s; 3 of
// up to 131072 112 us); a tile's weights, 1.3 us, and 1 to 2 us for a unit's begin and end and for each tile that rows see in part
// (48 requests with 5 new tokens, window 4096, fp32 results: 139 us, 5.3 TB/s).  The roles run side by side, so the code of all
// has to stay in the instruction cache: 94 KB took 178 us there, 85 KB 138.  Hence the rolled loops and the functions that
// are not inlined.
#include <cfloat>

#include "attn_paged.cuh"

namespace bl {
namespace {

using namespace attn;

template <int NR_>
struct TcShape {
  static constexpr int ROWS = NR_, TT = 128;
};

constexpr int kThreads = 16 * 32;
constexpr int kSlots = 5, kHalf = 128 * 256;  // bytes of 128 rows of k or v
constexpr int kBack = 4;                      // tiles whose pages, lists of odd values and sums of weights are kept
// Tiles whose descriptions are kept.  Warp 15 describes tile j when the copies of j - 4 are on their way; those waited for
// the product with v of j - 7, and that for the sums of j - 9: the sums of j - 8 may still read their tile's.
constexpr int kInfo = 16;
constexpr int kWeigh = 256;                   // threads of the weights
constexpr float kSlack = 8.f;                 // log2 of what a weight may be above 1

__host__ __device__ constexpr uint32_t tc_idesc(int n, bool a_m_major) {  // bf16 x bf16 -> fp32, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(a_m_major) << 15) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}
// M-major operand in the 128-byte swizzle: 64 values of M in 128 bytes, 8 rows of K in 1024; the next 64 of M lie
// `m_bytes` on.
__device__ __forceinline__ uint64_t tc_desc_m_major(uint32_t saddr, uint32_t m_bytes) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | uint64_t(m_bytes >> 4) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}

// A tile, for the warps that weigh it and add it up.
struct Tile {
  int j0, length, n;      // its first token; the request's tokens, and new ones
  Unit unit;
  int fresh, begun, ends; // the first tile of a unit or of the stretch; the unit's first is in the stretch; its last
  int left;               // tiles of the unit after this one
  int request, whole;     // every row sees all of its tokens, if they are there
  uint32_t real[4];       // tokens that are there
};

// A token of a tile whose value has infinities or NaN and that some rows do not see.
struct Odd {
  int token;              // of the tile
  uint32_t seen;          // by row: who sees it
};

template <int NR>
struct __align__(16) Tables {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t s_full[2], s_empty[2], o_full[2], o_empty[2], p_full, p_empty, voted[2], info[kBack], last;
  uint64_t found[kBack], taken[kBack];  // the pages of a tile
  uint64_t q_full[3];
  uint32_t tmem;
  unsigned dead;                 // a wait gave up
  int fills[kSlots];             // times that a slot's copies have been started
  Tile tile[kInfo];
  int block[kBack][16];          // the blocks of rows of a tile's pages in the caches
  int row[kBack];                // the first row in them
  float4 shift[NR / 4];          // maximum times scale
  float top[NR];                 // the maximum that weights are beside
  float part[4][NR];             // largest scores of the warps' tokens
  int vote[kBack];               // whether a score of the tile is far above it
  float4 keep[kBack][NR / 4];    // what the sums before the tile are multiplied by
  float sum[kBack][4][NR], final_top[kBack][NR];  // of a unit that ends (here) with the tile
  int odd_count[kBack];
  Odd odd[kBack][128];
  int64_t before[kThreads + 1];
  int64_t warp_total[kThreads / 32];
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}
// Folds v[0..15] over the 32 lanes: lane l gets op over all lanes of v[l % 16].
template <class Op>
__device__ __forceinline__ float fold(float (&v)[16], int lane, Op op) {
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = op(v[k], __shfl_xor_sync(0xffffffffu, v[k], 16));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const bool up = lane & o;
      const float mine = up ? v[k + o] : v[k], other = up ? v[k] : v[k + o];
      v[k] = op(mine, __shfl_xor_sync(0xffffffffu, other, o));
    }
  return v[0];
}

__device__ __forceinline__ bool odd_value(uint32_t u) { return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u; }

// The rest of a wait that did not end at once, out of line: the roles' loops have to share the instruction cache.  False: it
// gave up, or, unless `all`, another one has (`dead`); the role then ends, and touches nothing that it has not waited for.
// `all` is for the warps of the weights, which meet at barriers behind their vote: no look at `dead`, so that either all of
// them pass or none does.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, unsigned* dead, bool all) {
  const bool ok = (all || *static_cast<volatile unsigned*>(dead) == 0) && mbar_wait_bounded(bar, parity, nullptr);
  if (!ok) *static_cast<volatile unsigned*>(dead) = 1;
  return __all_sync(0xffffffffu, ok);
}

template <class S>
__device__ __noinline__ Place<S> first_tile(const Args& a, const int64_t* before, int64_t share, int64_t t0) {
  Place<S> at;
  at.find(a, before, kThreads, share, t0);
  return at;
}

template <int NR, bool F32>
__global__ void __launch_bounds__(kThreads, 1) attn_paged_tc_kernel(const Args a, const __grid_constant__ CUtensorMap k_map,
                                                                   const __grid_constant__ CUtensorMap v_map) {
  using S = TcShape<NR>;
  constexpr int PN = TERMS * NR;
  constexpr int kQBytes = NR * 256, kCols = 2 * NR + 2 * PN <= 128 ? 128 : 256;
  extern __shared__ uint8_t raw[];
  __shared__ Tables<NR> c;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* queries = ring + kSlots * kHalf;     // three units' q: [2][NR][64]
  uint8_t* weights = queries + 3 * kQBytes;     // [2][PN][64 tokens]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  auto wait = [&](uint64_t* bar, int parity, bool all = false) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, uint32_t(parity & 1))) || wait_on(bar, parity & 1, &c.dead, all);
  };

  if (warp == 14) {
    tmem_alloc(&c.tmem, kCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    c.dead = a.wait_ns != 0;  // a test limit: as if a wait had given up
#pragma unroll 1
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&c.full[i], 1);
      mbar_init(&c.empty[i], 1);
      c.fills[i] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.s_empty[i], 8);
      mbar_init(&c.o_full[i], 1);
      mbar_init(&c.o_empty[i], 4);
      mbar_init(&c.voted[i], 8);
    }
    for (int i = 0; i < kBack; ++i) {
      mbar_init(&c.info[i], 8);
      mbar_init(&c.found[i], 1);
      mbar_init(&c.taken[i], 2);
      c.vote[i] = 0;
      c.odd_count[i] = 0;
    }
    for (int i = 0; i < 3; ++i) mbar_init(&c.q_full[i], 32);
    mbar_init(&c.p_full, 8);
    mbar_init(&c.p_empty, 1);
    mbar_init(&c.last, 1);
    fence_barrier_init();
  }
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
    if (lane == 31) c.warp_total[warp] = through;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t sum = 0;
    for (int i = 0; i < warp; ++i) sum += c.warp_total[i];
    c.before[tid + 1] = sum + through;
    if (tid == 0) c.before[0] = 0;
    __syncthreads();
  }
  const uint32_t tmem = c.tmem;
  const int64_t all = c.before[kThreads];
  const int64_t quota = max(int64_t(1), quotient(all + gridDim.x - 1, gridDim.x));
  const int64_t t0 = blockIdx.x * quota;
  const int count = int(max(int64_t(0), min(quota, all - t0)));

  if (count > 0 && warp == 15) {
    // ---- ahead: a lane has four tokens of a tile ----
    Place<S> at = first_tile<S>(a, c.before, share, t0);
    // The page of token `k` of a tile as the table has it (not looked at before it is needed).
    auto page_of = [&](const Place<S>& pl, int k) {
      const int j = pl.token() + k;
      return j < pl.q.length ? a.table[pl.r * a.W + a.by_page.quotient(j)] : -1;
    };
    const int box_log = 31 - __clz(min(a.page, 128));
    int entry[4], then_entry[4];
    Place<S> then = at;  // the tile after this one, whose pages are looked up meanwhile
    bool fresh = true, begun = false;
#pragma unroll 1
    for (int i = -1; i < count; ++i) {
      if (i >= 0) {
#pragma unroll
        for (int h = 0; h < 4; ++h) entry[h] = then_entry[h];
        at = then;
        if (i + 1 < count) then.next(a);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) then_entry[h] = page_of(then, h * 32 + lane);
      if (i < 0) continue;
      const int buf = i % kBack;
      if (i >= kBack && !wait(&c.taken[buf], i / kBack - 1)) break;
      const int head = at.head(), row0 = at.row0(), j0 = at.token();
      Tile& info = c.tile[i % kInfo];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int k = h * 32 + lane, j = j0 + k;
        const bool seen = j < at.q.length && !(a.window > 0 && j < at.q.low && j >= a.sinks);  // by a row
        if (entry[h] < 0 || entry[h] >= a.pages) {
          bad |= seen;
          entry[h] = -1;
        }
        const unsigned there = __ballot_sync(0xffffffffu, seen && entry[h] >= 0);
        if (lane == 0) info.real[h] = there;
        // of the page's first token in the tile: the block, one behind the last where there is none
        const int off = j - a.by_page.quotient(j) * a.page;
        if (k == 0) c.row[buf] = off;
        if (k == 0 || off == 0) c.block[buf][k >> box_log] = entry[h] < 0 ? int(a.pages) * a.Hk : entry[h] * a.Hk + head;
      }
      if (fresh) begun = at.tile == 0;
      if (lane == 0) {
        info.j0 = j0;
        info.length = at.q.length;
        info.n = at.q.n;
        info.unit = {at.q.first, head, row0, int(min(int64_t(at.q.n) * a.G - row0, int64_t(NR)))};
        info.fresh = fresh;
        info.begun = begun;
        info.ends = at.tile + 1 == at.q.tiles;
        info.left = at.q.tiles - 1 - at.tile;
        info.request = int(at.r);
        info.whole = j0 + 127 <= at.q.length - at.q.n &&
                     (a.window <= 0 || j0 + 128 <= a.sinks || j0 > int64_t(at.q.length) - 1 - a.window);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.found[buf]);
      fresh = at.tile + 1 == at.q.tiles;
    }
  } else if (count > 0 && (warp == 12 || warp == 13)) {
    // ---- copies of k (and the queries) or v ----
    const int half = warp - 12;
    const int rows = min(a.page, 128), boxes = 128 / rows;
    const CUtensorMap* map = half ? &v_map : &k_map;
    int unit = -1;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const int buf = i % kBack, seq = 2 * i + half, slot = seq % kSlots;
      if (!wait(&c.found[buf], i / kBack)) break;
      const Tile& now = c.tile[i % kInfo];
      if (seq >= kSlots && !wait(&c.empty[slot], seq / kSlots - 1)) break;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(&c.full[slot], kHalf);
        c.fills[slot] = seq / kSlots + 1;
      }
      __syncwarp();
      // a lane per box of 64 columns of a page's rows
#pragma unroll 1
      for (int x = lane; x < 2 * boxes; x += 32)
        tma_load_3d(smem_addr(ring) + slot * kHalf + (x & 1) * (kHalf / 2) + (x >> 1) * rows * 128, map, (x & 1) * 64, c.row[buf], c.block[buf][x >> 1],
                    &c.full[slot]);
      if (half == 0 && now.fresh) {  // the unit's queries; the buffer's last reader was three units ago
        ++unit;
        const Unit u = now.unit;
#pragma unroll 1
        for (int k = lane; k < NR * 16; k += 32) {
          const int row = k / 16, ch = k % 16;
          const bool real = row < u.n && ch * 8 < a.D && !a.zero;
          copy16(smem_addr(queries) + (unit % 3) * kQBytes + (ch / 8) * (kQBytes / 2) + row * 128 + ((ch % 8) ^ (row & 7)) * 16,
                 a.q + (real ? row_at(a, u, row) + ch * 8 : 0), real);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&c.q_full[unit % 3])) : "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.taken[buf]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (count > 0 && warp == 14) {
    // ---- products: the next tile's scores are formed while this one's are weighed ----
    const uint64_t k_at = umma_desc_sw128(smem_addr(ring)), q_at = umma_desc_sw128(smem_addr(queries));
    const uint64_t v_at = tc_desc_m_major(smem_addr(ring), kHalf / 2), p_at = umma_desc_sw128(smem_addr(weights));
    int units = -1;
#pragma unroll 1
    for (int i = 0; i <= count; ++i) {
      if (i < count) {  // S(i)
        const int slot = 2 * i % kSlots;
        if (!wait(&c.full[slot], 2 * i / kSlots)) break;
        if (i >= 2 && !wait(&c.s_empty[i & 1], i / 2 - 1)) break;
        tc_fence_after();
        if (c.tile[i % kInfo].fresh) {
          ++units;
          if (!wait(&c.q_full[units % 3], units / 3)) break;
          fence_async_smem();  // the queries were copied by the generic proxy
          __syncwarp();
        }
        if (elect_one()) {
          const uint64_t k = k_at + slot * (kHalf >> 4), q = q_at + (units % 3) * (kQBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_f16(tmem + (i & 1) * NR, k + (ks / 4) * (kHalf >> 5) + (ks % 4) * 2, q + (ks / 4) * (kQBytes >> 5) + (ks % 4) * 2, tc_idesc(NR, false), ks > 0);
          umma_commit(&c.s_full[i & 1]);
          umma_commit(&c.empty[slot]);
        }
        __syncwarp();
      }
      if (i > 0) {  // O(i - 1)
        const int j = i - 1, slot = (2 * j + 1) % kSlots;
        if (!wait(&c.full[slot], (2 * j + 1) / kSlots)) break;
        if (j >= 2 && !wait(&c.o_empty[j & 1], j / 2 - 1)) break;
        if (!wait(&c.p_full, j)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t v = v_at + slot * (kHalf >> 4);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_f16(tmem + 2 * NR + (j & 1) * PN, v + ks * (16 * 128 >> 4), p_at + (ks / 4) * (PN * 128 >> 4) + (ks % 4) * 2, tc_idesc(PN, true), ks > 0);
          umma_commit(&c.o_full[j & 1]);
          umma_commit(&c.p_empty);
          umma_commit(&c.empty[slot]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) umma_commit(&c.last);
    __syncwarp();
  } else if (count > 0 && warp >= 8) {
    // ---- sums: thread t has coordinate t ----
    const int t = tid - 256;
    const uint32_t lanes = uint32_t(warp % 4 * 32) << 16;
    float acc[NR];
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const int buf = i % kBack;
      const Tile& was = c.tile[i % kInfo];
      if (!wait(&c.info[buf], i / kBack)) break;
      if (!wait(&c.o_full[i & 1], i / 2)) break;
      __syncwarp();
      tc_fence_after();
      if (was.fresh) {
#pragma unroll
        for (int r = 0; r < NR; ++r) acc[r] = 0.f;
      }
#pragma unroll
      for (int h = 0; h < NR; h += 16) {
        uint32_t u[TERMS][16];
        float o[16];
#pragma unroll
        for (int k = 0; k < TERMS; ++k) tmem_ld16(tmem + lanes + 2 * NR + (i & 1) * PN + k * NR + h, u[k]);
        tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          o[r] = __uint_as_float(u[TERMS - 1][r]);
#pragma unroll
          for (int k = TERMS - 2; k >= 0; --k) o[r] += __uint_as_float(u[k][r]);
        }
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const float4 keep = c.keep[buf][(h + r) / 4];
          acc[h + r] = __fmaf_rn(acc[h + r], keep.x, o[r]);
          acc[h + r + 1] = __fmaf_rn(acc[h + r + 1], keep.y, o[r + 1]);
          acc[h + r + 2] = __fmaf_rn(acc[h + r + 2], keep.z, o[r + 2]);
          acc[h + r + 3] = __fmaf_rn(acc[h + r + 3], keep.w, o[r + 3]);
        }
      }
      tc_fence_before();
      const int odd = c.odd_count[buf];
#pragma unroll 1
      for (int k = 0; k < odd; ++k) {
        const Odd x = c.odd[buf][k];
        const int j = was.j0 + x.token;
        const int64_t entry = a.table[was.request * a.W + a.by_page.quotient(j)];
        const float v = t < a.D ? bf16_bits_to_f32(a.v[((entry * a.Hk + was.unit.head) * a.page + j - a.by_page.quotient(j) * a.page) * a.D + t]) : 0.f;
        if (!(fabsf(v) < INFINITY)) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
            acc[r] += x.seen >> r & 1 ? v : 0.f;  // times a weight above 0
        }
      }
      if (was.ends || i + 1 == count) {
        // A lane has a row's sum of weights, and where the row goes: to the result, or to the workspace as a part.
        static_assert(NR == 32, "a lane per row");
        const bool out = was.begun && was.ends;
        const int64_t part = 2 * int64_t(blockIdx.x) + was.begun;
        const int n = was.unit.n;
        const float l = (c.sum[buf][0][lane] + c.sum[buf][1][lane]) + (c.sum[buf][2][lane] + c.sum[buf][3][lane]);
        const float top = c.final_top[buf][lane];
        const float inv = !out ? 1.f : top == -INFINITY && l == 0.f ? 0.f : 1.f / l;
        const int64_t first = out ? row_at(a, was.unit, 0) : part * a.rows * a.D;
        const int mine = !out ? lane * a.D : lane < n ? int(row_at(a, was.unit, lane) - first) : 0;
        if (!out && warp == 8 && lane < n) a.stat[part * a.rows + lane] = make_float2(top, l);
        const int end = t < a.D ? n : 0;
        auto each_row = [&](auto store) {
#pragma unroll 1
          for (int row = 0; row < NR; row += 8) {  // eight at a time, the next ones moved to their place: little code
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const int to = __shfl_sync(0xffffffffu, mine, row + r);
              const float by = __shfl_sync(0xffffffffu, inv, row + r);
              store(to, acc[r] * by, row + r < end);
            }
#pragma unroll
            for (int r = 0; r + 8 < NR; ++r) acc[r] = acc[r + 8];
          }
        };
        if (F32 || !out) {
          float* sums = (out ? static_cast<float*>(a.out) : a.acc) + first + t;
          each_row([&](int to, float v, bool real) {
            asm volatile("{.reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.f32 [%0], %1;}" ::"l"(sums + to), "f"(v), "r"(unsigned(real)) : "memory");
          });
        } else {
          uint16_t* sums = static_cast<uint16_t*>(a.out) + first + t;
          each_row([&](int to, float v, bool real) {
            asm volatile("{.reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.u16 [%0], %1;}" ::"l"(sums + to), "h"(f32_to_bf16_bits_rn(v)), "r"(unsigned(real))
                         : "memory");
          });
        }
        if (t == 0 && i + 1 == count) {
          Header header = {};
          if (was.begun && !was.ends) header = Header{was.unit, 1, int(quotient(t0 + i + was.left, quota) - blockIdx.x), {0, 0}};
          a.header[blockIdx.x] = header;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.o_empty[i & 1]);  // of the tile's tables too
    }
  } else if (count > 0) {
    // ---- weights: thread t % 128 has a token of a tile, and 16 of the rows ----
    static_assert(NR == 32, "16 rows to a thread");
    constexpr int HR = 16;
    const int t = tid % 128, first_row = tid / 128 * HR;
    const uint32_t lanes = uint32_t(warp % 4 * 32) << 16;
    const uint32_t flip = a.sign & 0x80000000u;
    // where this lane stores weights: of tokens t & ~1 and t | 1, of the rows 4, 5, 6, 7 beyond every eight for odd lanes
    const uint32_t p_to = smem_addr(weights) + first_row * 128 + (t / 64) * (PN * 128) + (t % 8 & 6) * 2;
    const uint32_t p_chunk = t % 64 / 8;
    const bool up = lane & 1;
    float sum[HR];
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const int buf = i % kBack;
      if (!wait(&c.s_full[i & 1], i / 2)) break;
      __syncwarp();
      tc_fence_after();
      uint32_t zu[HR];
      tmem_ld16(tmem + lanes + (i & 1) * NR + first_row, zu);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.s_empty[i & 1]);
      const Tile& now = c.tile[i % kInfo];
      const int j = now.j0 + t, nrows = now.unit.n;
      const bool fresh = now.fresh;
      float z[HR];
#pragma unroll
      for (int r = 0; r < HR; ++r) z[r] = __uint_as_float(zu[r] ^ flip);
      const unsigned there = now.real[warp % 4];
      const bool whole = now.whole && (now.real[0] & now.real[1] & now.real[2] & now.real[3]) == 0xffffffffu;
      // Which rows see the token: those from its own new token on, up to the one whose window it has left.
      const uint32_t rows_mask = nrows >= 32 ? 0xffffffffu : (1u << nrows) - 1;
      uint32_t seen = rows_mask;
      if (!whole) {
        const int first_new = now.length - now.n;
        const int from = max(0, min(j - first_new, now.n)) * a.G - now.unit.row0;
        const bool bounded = a.window > 0 && j >= a.sinks;
        const int end = (bounded ? int(max(int64_t(0), min(j + a.window - first_new, int64_t(now.n)))) : now.n) * a.G - now.unit.row0;
        auto below = [](int r) { return r >= 32 ? 0xffffffffu : r <= 0 ? 0u : (1u << r) - 1; };
        seen &= there >> lane & 1 ? below(end) & ~below(from) : 0u;
#pragma unroll
        for (int r = 0; r < HR; ++r) z[r] = seen >> (first_row + r) & 1 ? z[r] : -INFINITY;
      }
      const bool partly = seen != rows_mask;
      // Weights beside the maximum as it was; a unit's first tile has none yet.
      float p[HR];
      auto weigh = [&]() {
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
          const float4 shift = c.shift[(first_row + r) / 4];
          p[r] = __fmaf_rn(z[r], a.scale, -shift.x);
          p[r + 1] = __fmaf_rn(z[r + 1], a.scale, -shift.y);
          p[r + 2] = __fmaf_rn(z[r + 2], a.scale, -shift.z);
          p[r + 3] = __fmaf_rn(z[r + 3], a.scale, -shift.w);
        }
        float most = p[0];
#pragma unroll
        for (int r = 1; r < HR; ++r) most = fmaxf(most, p[r]);
#pragma unroll
        for (int r = 0; r < HR; ++r) p[r] = exp2_fast(p[r]);
        return most;
      };
      const bool far = fresh || weigh() > kSlack;
      if (__any_sync(0xffffffffu, far) && lane == 0) c.vote[buf] = 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.voted[i & 1]);
      if (!wait(&c.voted[i & 1], i / 2, true)) break;  // all eight warps or none: barriers follow
      const bool rises = c.vote[buf] != 0;
      if (__builtin_expect(rises, 0)) {
        float v[HR];
#pragma unroll
        for (int r = 0; r < HR; ++r) v[r] = z[r];
        const float most = fold(v, lane, [](float x, float y) { return fmaxf(x, y); });
        if (lane < HR) c.part[warp % 4][first_row + lane] = most;
        named_barrier_sync(2, kWeigh);
        if (tid < NR) {
          const float old = fresh ? -INFINITY : c.top[tid];
          const float top = fmaxf(fmaxf(fmaxf(c.part[0][tid], c.part[1][tid]), fmaxf(c.part[2][tid], c.part[3][tid])), old);
          // A row that has seen nothing: what it does not see keeps a weight of 0, and the first score that it sees lies far
          // above -FLT_MAX, whatever its size, and raises the maximum.  Rows behind the unit's last have none to raise.
          const bool none = top == -INFINITY;
          c.top[tid] = top;
          reinterpret_cast<float*>(c.shift)[tid] = !none ? top * a.scale : tid < nrows ? -FLT_MAX : 0.f;
          reinterpret_cast<float*>(c.keep[buf])[tid] = none ? 0.f : exp2_fast((old - top) * a.scale);
        }
        named_barrier_sync(2, kWeigh);
        weigh();
#pragma unroll
        for (int r = 0; r < HR; ++r) sum[r] = fresh ? p[r] : __fmaf_rn(sum[r], reinterpret_cast<const float*>(c.keep[buf])[first_row + r], p[r]);
      } else {
#pragma unroll
        for (int r = 0; r < HR; ++r) sum[r] += p[r];
      }
      if (!rises && tid < NR) reinterpret_cast<float*>(c.keep[buf])[tid] = 1.f;
      if (tid == 0) c.vote[(i + 2) % kBack] = 0;
      if (i > 0 && !wait(&c.p_empty, i - 1)) break;
      __syncwarp();
      if (tid == 0) c.odd_count[(i + 1) % kBack] = 0;
      // Two lanes exchange rows, so that each stores a pair of tokens; rows r and r + 4 lie in different banks.
#pragma unroll
      for (int k = 0; k < HR / 2; ++k) {
        const int r = k / 4 * 8 + k % 4;
        const float other = __shfl_xor_sync(0xffffffffu, up ? p[r] : p[r + 4], 1);
        float lo = up ? other : p[r], hi = up ? p[r + 4] : other;
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          const int row = term * NR + r;
          const uint32_t u = bf16x2_rn(lo, hi);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(p_to + (up ? (row + 4) * 128 + ((p_chunk ^ ((r + 4) & 7)) * 16) : row * 128 + ((p_chunk ^ (r & 7)) * 16))),
                       "r"(u)
                       : "memory");
          lo -= __uint_as_float(u << 16);
          hi -= __uint_as_float(u & 0xffff0000u);
        }
      }
      // A value that some rows do not see (or none: the rest of a page) must not reach them, and 0 times an infinity or
      // NaN would: such values are taken out of the tile, and added to the sums of the rows that see them.
      if (__builtin_expect(__any_sync(0xffffffffu, partly), 0)) {
        const int seq = 2 * i + 1, slot = seq % kSlots;
        if (!wait(&c.full[slot], seq / kSlots)) break;
        __syncwarp();
        if (partly && first_row == 0) {  // the other half of the rows leaves it to this thread
          bool odd = false;
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {  // lanes begin at different banks
            const uint32_t v = smem_addr(ring) + slot * kHalf + (k / 8) * (kHalf / 2) + t * 128 + ((k ^ t) % 8) * 16;
            uint32_t u[4];
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(v) : "memory");
            if (odd_value(u[0]) || odd_value(u[1]) || odd_value(u[2]) || odd_value(u[3])) {
              odd = true;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((u[e] & 0x7f80u) == 0x7f80u) u[e] &= 0xffff0000u;
                if ((u[e] & 0x7f800000u) == 0x7f800000u) u[e] &= 0x0000ffffu;
              }
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(v), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
            }
          }
          if (odd && seen) c.odd[buf][atomicAdd(&c.odd_count[buf], 1)] = Odd{t, seen};
        }
      }
      if (__builtin_expect(now.ends || i + 1 == count, 0)) {
        float v[HR];
#pragma unroll
        for (int r = 0; r < HR; ++r) v[r] = sum[r];
        const float total = fold(v, lane, [](float x, float y) { return x + y; });
        if (lane < HR) {
          c.sum[buf][warp % 4][first_row + lane] = total;
          if (warp % 4 == 0) c.final_top[buf][first_row + lane] = c.top[first_row + lane];
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&c.p_full);
        mbar_arrive(&c.info[buf]);
      }
    }
  } else if (count == 0 && tid == 0) {
    a.header[blockIdx.x] = Header{};
  }
  if (count > 0 && warp == 14) mbar_wait_bounded(&c.last, 0, nullptr);  // no product is in flight
  __syncwarp();
  if (__syncthreads_or(bad) && tid == 0) atomicOr(a.err, BL_DEVERR_RANGE);
  if (c.dead) {  // copies may still be in flight: they land before the CTA ends; no unit goes on from here
    if (tid < kSlots && c.fills[tid] > 0) mbar_wait_bounded(&c.full[tid], (c.fills[tid] - 1) & 1, nullptr);
    if (tid == 0) {
      atomicOr(a.err, BL_DEVERR_WAIT_TIMEOUT);
      a.header[blockIdx.x] = Header{};
    }
    __syncthreads();
  }
  if (warp == 14) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  pdl_launch_dependents();
}

template <int NR, bool F32>
cudaError_t launch_as(const Args& a, const CUtensorMap& k_map, const CUtensorMap& v_map, int grid, cudaStream_t s) {
  constexpr int kBytes = 1024 + kSlots * kHalf + 3 * NR * 256 + TERMS * NR * 256;
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t e = raise_smem_cap(attn_paged_tc_kernel<NR, F32>, dev, kBytes);
  if (e != cudaSuccess) return e;
  return launch(attn_paged_tc_kernel<NR, F32>, dim3(grid), dim3(kThreads), kBytes, s, overlap_enabled(), a, k_map, v_map);
}

}  // namespace

namespace attn {

cudaError_t launch_tc(const Args& a, int grid, bool f32, cudaStream_t s) {
  const bool whole = a.page % 128 == 0 || (a.page < 128 && a.page >= 8 && 128 % a.page == 0);
  CUtensorMap k_map, v_map;
  const uint64_t blocks = uint64_t(a.pages) * a.Hk;
  // (a unit's rows are found by 32-bit offsets)
  if (!whole || blocks >= 0x7fffffff || int64_t(a.H) * a.D > 1 << 25 ||
      !encode_tmap_blocks_bf16(&k_map, a.k, a.D, a.page, blocks, 64, std::min(a.page, 128)) ||
      !encode_tmap_blocks_bf16(&v_map, a.v, a.D, a.page, blocks, 64, std::min(a.page, 128)))
    return cudaErrorNotSupported;
  return f32 ? launch_as<32, true>(a, k_map, v_map, grid, s) : launch_as<32, false>(a, k_map, v_map, grid, s);
}

}  // namespace attn
}  // namespace bl
