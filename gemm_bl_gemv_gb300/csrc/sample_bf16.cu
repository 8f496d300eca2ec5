// Sampling from bf16 logits (bl_sample).  A row has at most 65281 different
// live values, so a histogram over the 16-bit keys says everything: one
// weight per different value times an exact count, and the order of the
// tokens is the order of the bins.  No exp per logit, one shared-memory
// atomic per logit.
//
// A cluster of C CTAs takes a row, each CTA a chunk of it.  Word i of a CTA's
// histogram (128 KB) counts the positive logits of magnitude bits i in its
// low half and the negative ones in its high half, so a logit finds its
// counter without being turned into a key.  A counter holds 16 bits: before
// one could overflow, a chunk of more than 65535 logits looks for the largest
// counter and moves what is above half of the range to a short list.  The
// bins are cut into 1024 segments of 64; only the segments that some CTA has
// hit (some tens, of a model's logits) are weighed, one warp each, with the
// counts of all C histograms read through distributed shared memory.  One
// warp of the first CTA then finds the places in the order: first the segment
// in which a cumulative count or weight passes the goal, then the bin.  The
// CTA whose chunk has the token looks up its index while the next row's
// places are found.  Clusters stay for several rows and clear only the segments
// that they hit.
//
// Bound: a random shared-memory atomic takes 3.5 clocks per warp (bank
// conflicts, as a plain load's; measured), 23 us for 256 rows of 248320 logits
// on 152 SMs, whose bytes take 18.7 us at the copy rate; beside it each row has
// some 8 us of dependent steps (weights of the segments, places, the look-up).
// 256 rows of 248320: 74 us, two rounds; 64 rows: 27 us; one row: 19 us, the
// exchanges of a cluster of 8.
#include "sample_common.cuh"

namespace bl {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kWords = 32768;                // counters of one magnitude: low half positive, high half negative
constexpr int kSegments = 1024;              // 64 magnitudes of one sign each, in falling order
constexpr int kStep = 2000;                  // groups counted at a time, two per thread: four steps fit in 2^16 - 16 logits
constexpr int kBatch = 128;                  // groups of 8 logits that a warp looks through at a time
constexpr int kSpills = 32;                  // at most 524288 / 32767 counters are moved
constexpr uint32_t kMasked2 = 0xFF80FF80u;   // two logits of -inf
constexpr uint32_t kInf = 0x7F80u;           // magnitude bits of an infinity; above: NaN
// weights below 2^-45 of the largest are 0: no bin further than 46 octaves (31.9 T) matters
constexpr float kWindow = 32.f;

using Args = SampleArgs;

// A place in the order: the logit of these bf16 bits with `rank` equal ones
// before it; `before` is the weight of everything before those.
struct Place {
  uint32_t bits;
  u64 rank, before, weight;
};

// A segment with the sums over all CTAs.  index: its place among the 1024,
// 0..511 positive (magnitudes falling), 512..1023 negative (rising).
struct Segment {
  u64 mass;
  uint32_t count, index;
};

struct Spill {
  uint32_t bits, count;
};

// What the lookup of a token's index needs, kept until the next row's search.
struct Pick {
  uint32_t bits, rank;
  u64 kept;
  float top;
  Slope slope;
};

struct Shared {
  uint32_t hist[kWords];
  // read by the other CTAs of the cluster
  uint16_t bitmap[64];  // segments that this CTA has hit: 16 positive per entry (rising), then 16 negative per entry
  uint32_t top;         // its largest live logit's bits + 1, 0 if there is none
  uint32_t spills;      // counters moved to the list
  Spill spill[kSpills];
  // written by the other CTAs (to rank 0's), in falling order
  Segment seg[kSegments];
  // written by rank 0
  uint32_t pick_bits, pick_rank, pick_owner;
  u64 kept;
  // local
  u64 mass_before[kSegments];
  uint32_t count_before[kSegments];
  Exp2Table exp2;
  Pick pick;
  uint32_t warp_max[kWarps];
  uint32_t matches[2][2 * kWarps];  // by batch of a round
};

__device__ __forceinline__ float value_of(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint32_t order_of(uint32_t bits) {  // rises with the value
  return (bits & 0x8000u) ? 0xFFFFu - bits : bits | 0x8000u;
}

// Count a logit whose bits are the upper half of `w`, at byte offset `at` of
// the histogram; -inf and negative NaN are left out (a mask would put them all
// on one address), positive NaN are cleared later.  A predicated instruction:
// a branch around each atomic costs more than the atomic.
__device__ __forceinline__ void count_logit(uint32_t hist, uint32_t w, uint32_t at) {
  asm volatile(
      "{\n\t.reg .pred live, neg;\n\t.reg .u32 one;\n\t"
      "setp.lt.u32 live, %0, 0xFF800000;\n\t"
      "setp.lt.s32 neg, %0, 0;\n\t"
      "selp.u32 one, 0x10000, 1, neg;\n\t"
      "@live red.shared.add.u32 [%1], one;\n\t}" ::"r"(w),
      "r"(hist + at)
      : "memory");
}
__device__ __forceinline__ void count_pair(uint32_t hist, uint32_t w) {
  count_logit(hist, w << 16, (w << 2) & 0x1FFFCu);
  count_logit(hist, w, (w >> 14) & 0x1FFFCu);
}
__device__ __forceinline__ void count_group(uint32_t hist, uint4 q) {
  count_pair(hist, q.x);
  count_pair(hist, q.y);
  count_pair(hist, q.z);
  count_pair(hist, q.w);
}

// The logits of one value.
struct Target {
  uint32_t two, mask;  // in both halves; -0 equals 0
  __device__ __forceinline__ explicit Target(uint32_t bits)
      : two(bits | bits << 16), mask(bits == 0 ? 0x7FFF7FFFu : 0xFFFFFFFFu) {}
  __device__ __forceinline__ uint32_t in(uint32_t w) const {
    const uint32_t t = (w ^ two) & mask;
    return uint32_t((t & 0xFFFFu) == 0) | uint32_t((t >> 16) == 0) << 1;
  }
  // bit j: logit j of the group has the value; most groups fail the quick test (a zero half of w ^ target)
  __device__ __forceinline__ uint32_t in(const uint4& q) const {
    auto zero = [&](uint32_t w) {
      const uint32_t t = (w ^ two) & mask;
      return (t - 0x00010001u) & ~t;
    };
    if (((zero(q.x) | zero(q.y) | zero(q.z) | zero(q.w)) & 0x80008000u) == 0) return 0;
    return in(q.x) | in(q.y) << 2 | in(q.z) << 4 | in(q.w) << 6;
  }
};

// The live segments of a row in falling order, held by a warp: lane i has
// segments 32 i .. 32 i + 31, from the highest bit down.
struct SegmentList {
  uint32_t bits, upto;  // segments of this lane; of this lane and those before it
  int n;
  __device__ __forceinline__ SegmentList(uint32_t word, int lane) {
    bits = word;
    upto = warp_scan(uint32_t(__popc(word)));
    n = int(__shfl_sync(0xffffffffu, upto, 31));
  }
  // The idx-th segment, idx < n (whole warp).
  __device__ __forceinline__ uint32_t at(uint32_t idx, int lane) const {
    const int src = __ffs(__ballot_sync(0xffffffffu, upto > idx)) - 1;
    const uint32_t w = __shfl_sync(0xffffffffu, bits, src);
    const uint32_t r = idx + __popc(w) - __shfl_sync(0xffffffffu, upto, src);
    // lane b looks at bit 31 - b
    const uint32_t above = lane == 0 ? 0u : w >> (32 - lane);
    const bool here = ((w >> (31 - lane)) & 1u) && __popc(above) == int(r);
    return 32u * src + __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  }
};

// Of a bitmap (Shared::bitmap), lane i's word of a SegmentList.
__device__ __forceinline__ uint32_t list_word(const uint16_t* bitmap, int lane) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(bitmap);
  return lane < 16 ? w[15 - lane] : __brev(w[lane]);
}

template <int C>
struct Row {
  Shared& sh;
  int lane;
  float top;
  Slope slope;
  int n;        // live segments
  bool spills;  // some CTA has moved counters

  __device__ __forceinline__ u64 weight(uint32_t bits) const { return weight_of(value_of(bits), top, slope, sh.exp2); }

  // This lane's two bins of a segment, in falling order.
  struct Bins {
    uint32_t bits1, bits0, c1, c0;
    u64 w1, w0;
  };
  __device__ __forceinline__ Bins bins(uint32_t seg) const {
    Bins b;
    const bool neg = seg >= 512;
    const uint32_t word = neg ? (seg - 512) * 64 + 2 * lane : (511 - seg) * 64 + 62 - 2 * lane;  // of two
    b.c1 = b.c0 = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const uint2* mine = reinterpret_cast<uint2*>(&sh.hist[word]);
      const uint2 v = *(C == 1 ? mine : peer(mine, r));
      b.c1 += neg ? v.x >> 16 : v.y & 0xFFFFu;
      b.c0 += neg ? v.y >> 16 : v.x & 0xFFFFu;
    }
    b.bits1 = neg ? 0x8000u + word : word + 1;
    b.bits0 = neg ? 0x8001u + word : word;
    if (spills) {
      for (int r = 0; r < C; ++r) {
        const uint32_t moved = *(C == 1 ? &sh.spills : peer(&sh.spills, r));
        for (uint32_t i = 0; i < moved; ++i) {
          const Spill e = *(C == 1 ? &sh.spill[i] : peer(&sh.spill[i], r));
          b.c1 += e.bits == b.bits1 ? e.count : 0;
          b.c0 += e.bits == b.bits0 ? e.count : 0;
        }
      }
    }
    b.w1 = weight(b.bits1);
    b.w0 = weight(b.bits0);
    return b;
  }

  // The place where the cumulative count or weight first exceeds `goal` (less
  // than the whole); whole warp.
  __device__ __forceinline__ Place find(bool by_count, u64 goal) const {
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      bool here = false;
      if (i < n) {
        const u64 at = by_count ? sh.count_before[i] : sh.mass_before[i];
        here = at <= goal && goal - at < (by_count ? sh.seg[i].count : sh.seg[i].mass);
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, here);
      if (!hit) continue;
      const int s = i0 + __ffs(hit) - 1;
      const Bins b = bins(sh.seg[s].index);
      const u64 m1 = b.c1 * b.w1, m0 = b.c0 * b.w0;
      const u64 cm = warp_scan(m1 + m0);
      const uint32_t cc = warp_scan(b.c1 + b.c0);
      const u64 before = sh.mass_before[s] + cm - m1 - m0;
      const u64 at = by_count ? u64(sh.count_before[s]) + cc - b.c1 - b.c0 : before;
      const u64 n1 = by_count ? b.c1 : m1, n0 = by_count ? b.c0 : m0;
      const bool in1 = at <= goal && goal - at < n1;
      const bool in0 = at + n1 <= goal && goal - at - n1 < n0;
      Place p{};
      if (in1) p = Place{b.bits1, by_count ? goal - at : (goal - at) / b.w1, before, b.w1};
      if (in0) p = Place{b.bits0, by_count ? goal - at - n1 : (goal - at - n1) / b.w0, before + m1, b.w0};
      const int src = __ffs(__ballot_sync(0xffffffffu, in1 || in0)) - 1;
      p.bits = __shfl_sync(0xffffffffu, p.bits, src);
      p.rank = __shfl_sync(0xffffffffu, p.rank, src);
      p.before = __shfl_sync(0xffffffffu, p.before, src);
      p.weight = __shfl_sync(0xffffffffu, p.weight, src);
      return p;
    }
    return Place{};
  }

  // Weight of the bins that weigh at least `min_w`: whole segments, and a part of one; whole warp.
  __device__ __forceinline__ u64 mass_from(u64 min_w) const {
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t seg = i < n ? sh.seg[i].index : 0;
      // its smallest value's bits (of finite ones)
      const uint32_t last = seg < 512 ? (511 - seg) * 64 : 0x8000u + min((seg - 512) * 64 + 63, kInf - 1);
      const bool less = i < n && weight(last) < min_w;
      const uint32_t hit = __ballot_sync(0xffffffffu, less);
      if (!hit) continue;
      const int s = i0 + __ffs(hit) - 1;
      const Bins b = bins(sh.seg[s].index);
      return sh.mass_before[s] + warp_sum_u64((b.w1 >= min_w ? b.c1 * b.w1 : 0) + (b.w0 >= min_w ? b.c0 * b.w0 : 0));
    }
    return sh.mass_before[n - 1] + sh.seg[n - 1].mass;
  }
};

// A CTA's part of a row: groups of 8 logits that are aligned in memory.  The
// row starts at element `off` of group 0 and ends before element `end`; of the
// chunk's groups [g0, g1), [ga, gb) are whole.
struct Chunk {
  const uint16_t* row16;
  int off, end, g0, g1, ga, gb;
  __device__ __forceinline__ Chunk(const uint16_t* row, int V, int rank, int groups) {
    off = int((reinterpret_cast<uintptr_t>(row) >> 1) & 7);
    row16 = row - off;
    end = off + V;
    g0 = rank * groups;
    g1 = min(g0 + groups, (end + 7) / 8);
    ga = max(g0, (off + 7) / 8);
    gb = min(g1, end / 8);
  }
  __device__ __forceinline__ uint4 whole(int i) const { return reinterpret_cast<const uint4*>(row16)[i]; }
  // Any group of the chunk: logits outside the row, and groups outside the chunk, are `other`.
  __device__ __forceinline__ uint4 group(int i, uint32_t other) const {
    if (i >= ga && i < gb) return whole(i);
    uint32_t w[4] = {other, other, other, other};
    if (i >= g0 && i < g1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = i * 8 + j;
        if (e >= off && e < end) w[j >> 1] = __byte_perm(w[j >> 1], row16[e], (j & 1) ? 0x5410 : 0x3254);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The index of the logit of row m of value `bits` with `rank` equal ones before
// it in the chunk (Shared::pick), by warps 1.. of the CTA: matches are counted
// by batches of groups, and one warp walks the batch that has it.
__device__ __forceinline__ void look_up(const Args& g, Shared& sh, int64_t m, int rank) {
  constexpr int kPickWarps = kWarps - 1;
  const int lane = threadIdx.x & 31, warp = int(threadIdx.x >> 5) - 1;
  const Chunk c(static_cast<const uint16_t*>(g.logits) + m * g.V, int(g.V), rank, g.chunk / 8);
  const Target target(sh.pick.bits);
  uint32_t left = sh.pick.rank;
  // rounds of two batches per warp, in order, until the matches suffice
  constexpr int kRound = 2 * kPickWarps;
  for (int b0 = 0;; b0 += kRound) {
    uint4 q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = c.g0 + (b0 + warp + (j >> 2) * kPickWarps) * kBatch + (j & 3) * 32 + lane;
      q[j] = i >= c.ga && i < c.gb ? c.whole(i) : make_uint4(~target.two, ~target.two, ~target.two, ~target.two);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int first = c.g0 + (b0 + warp + h * kPickWarps) * kBatch;
      int n = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) n += __popc(target.in(q[4 * h + j]));
      // parts of groups: only the chunk's first and last group can be one
      const int edge = lane == 0 ? c.g0 : c.g1 - 1;
      if (lane < 2 && (lane == 0 || edge > c.g0) && edge >= first && edge < first + kBatch &&
          (edge < c.ga || edge >= c.gb))
        n += __popc(target.in(c.group(edge, ~target.two)));
      n = redux_add(n);
      if (lane == 0) sh.matches[(b0 / kRound) & 1][warp + h * kPickWarps] = n;
    }
    named_barrier_sync(1, 32 * kPickWarps);
    const uint32_t* counts = sh.matches[(b0 / kRound) & 1];  // the other half is for the next round
    const uint32_t n0 = counts[2 * lane < kRound ? 2 * lane : 0] * (2 * lane < kRound);
    const uint32_t n1 = counts[2 * lane < kRound ? 2 * lane + 1 : 0] * (2 * lane < kRound);
    const uint32_t all = uint32_t(redux_add(int(n0 + n1)));
    if (left >= all && c.g0 + (b0 + kRound) * kBatch < c.g1) {
      left -= all;
      continue;
    }
    if (warp != 0) return;
    const uint32_t upto = warp_scan(n0 + n1);
    const int src = __ffs(__ballot_sync(0xffffffffu, upto > left)) - 1;
    left -= __shfl_sync(0xffffffffu, upto - n0 - n1, src);
    const uint32_t half = __shfl_sync(0xffffffffu, n0, src);
    const int batch = b0 + 2 * src + (left >= half);
    left -= left >= half ? half : 0;
    const int first = c.g0 + batch * kBatch + lane;
    uint32_t hits = 0;  // of this lane's four groups
#pragma unroll
    for (int j = 0; j < 4; ++j) hits |= target.in(c.group(first + 32 * j, ~target.two)) << (8 * j);
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      uint32_t bits = (hits >> (8 * j)) & 0xFFu;
      const uint32_t incl = warp_scan(uint32_t(__popc(bits)));
      const uint32_t here = __shfl_sync(0xffffffffu, incl, 31), excl = incl - __popc(bits);
      if (left >= excl && left < incl) {
        for (uint32_t e = left - excl; e > 0; --e) bits &= bits - 1;
        const Pick& p = sh.pick;
        g.token[m] = (first + 32 * j) * 8 + (__ffs(bits) - 1) - c.off;
        if (g.prob) g.prob[m] = share_of(value_of(p.bits), p.top, p.slope, sh.exp2, p.kept);
      }
      if (left < here) break;
      left -= here;
    }
    return;
  }
}

// The largest counter of the CTA's histogram; counters of at least 2^15 are
// moved to the list but for 1, so it stays below 2^15.  Whole CTA; ends with a
// barrier.
__device__ __forceinline__ uint32_t largest_counter(Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t most = 0;
#pragma unroll
  for (int q = 0; q < kWords / 4 / kThreads; ++q) {
    const uint4 v = reinterpret_cast<const uint4*>(sh.hist)[q * kThreads + threadIdx.x];
    most = __vmaxu2(most, __vmaxu2(__vmaxu2(v.x, v.y), __vmaxu2(v.z, v.w)));
  }
  uint32_t mine = max(most & 0xFFFFu, most >> 16);
  if (mine >= 0x8000u) {  // few threads, rarely
    for (int q = 0; q < kWords / kThreads; ++q) {
      const uint32_t magnitude = (q / 4 * kThreads + threadIdx.x) * 4 + q % 4;
      uint32_t w = sh.hist[magnitude];
      for (int sign = 0; sign < 2; ++sign) {
        const uint32_t n = (w >> (16 * sign)) & 0xFFFFu;
        if (n < 0x8000u) continue;
        w -= (n - 1) << (16 * sign);
        if (magnitude > kInf) continue;  // NaN
        const uint32_t i = atomicAdd(&sh.spills, 1u);  // at most 524288 / 32767 times
        sh.spill[i] = Spill{magnitude == 0 ? 0u : magnitude | sign << 15, n - 1};
      }
      sh.hist[magnitude] = w;
    }
    mine = 0x7FFFu;
  }
  mine = redux_max_u32(mine);
  if (lane == 0) sh.warp_max[warp] = mine;
  __syncthreads();
  mine = redux_max_u32(sh.warp_max[lane]);
  __syncthreads();
  return mine;
}

template <int C>
__global__ void __launch_bounds__(kThreads) sample_bf16_kernel(const Args g) {
  extern __shared__ uint4 smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const uint32_t rank = C == 1 ? 0 : cluster_ctarank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4* hist4 = reinterpret_cast<uint4*>(sh.hist);
  const uint32_t hist = smem_addr(sh.hist);
  for (int i = threadIdx.x; i < kWords / 4; i += kThreads) hist4[i] = make_uint4(0, 0, 0, 0);
  fill_exp2_table(sh.exp2);
  if (threadIdx.x == 0) sh.spills = 0;
  int64_t pick_row = -1;  // the row whose token is in this CTA's chunk and still to be looked up
  pdl_wait();
  __syncthreads();

  for (int64_t m = blockIdx.x / C; m < g.M; m += gridDim.x / C) {
    const RowValues values(m, g.temperature, g.top_k, g.top_p, g.min_p, g.u);
    const uint16_t* row = static_cast<const uint16_t*>(g.logits) + m * g.V;
    const Chunk c(row, int(g.V), int(rank), g.chunk / 8);

    // histogram; the row's first and last part of a group by one thread each
    if (threadIdx.x < 2) {
      const int part = threadIdx.x == 0 ? 0 : c.end / 8;
      if ((part < c.ga || part >= c.gb) && (threadIdx.x == 0 || part > 0))
        count_group(hist, c.group(part, kMasked2));
    }
    uint4 now[2], next[2];
    auto fetch = [&](uint4 (&q)[2], int from) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = from + j * kThreads + int(threadIdx.x);
        q[j] = i < min(c.gb, from + kStep) ? c.whole(i) : make_uint4(kMasked2, kMasked2, kMasked2, kMasked2);
      }
    };
    fetch(now, c.ga);
    int room = 65535 - 16;  // logits that cannot overflow a counter
    for (int from = c.ga; from < c.gb; from += kStep) {
      fetch(next, from + kStep);
      if (room < 8 * kStep) {
        __syncthreads();
        room = 65535 - int(largest_counter(sh));
      }
      room -= 8 * kStep;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        count_group(hist, now[j]);
        now[j] = next[j];
      }
    }
    const RowFilter f = row_filter(values, g.V);
    __syncthreads();
    // -0 counts as 0; no NaN; which segments were hit: a lane looks through half of one (8 x 16
    // bytes, from a start that keeps the lanes on different banks), a warp through 16 of both signs
    {
      uint32_t any = 0;
      const int half = (warp * 16 + (lane & 15)) * 16 + (lane >> 4) * 8;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int at = half + ((q + lane) & 7);
        uint4 v = hist4[at];
        if (at == 0) {
          v.x = (v.x & 0xFFFFu) + (v.x >> 16);
          if (v.x > 0xFFFFu) {
            sh.spill[atomicAdd(&sh.spills, 1u)] = Spill{0u, v.x - 1};
            v.x = 1;
          }
          sh.hist[0] = v.x;
        }
        if (at >= int(kInf) / 4) {
          v.x = at == int(kInf) / 4 ? v.x & 0xFFFFu : 0u;
          v.y = v.z = v.w = 0;
          hist4[at] = v;
        }
        any |= v.x | v.y | v.z | v.w;
      }
      any |= __shfl_xor_sync(0xffffffffu, any, 16);
      const uint32_t bl = __ballot_sync(0xffffffffu, (any & 0xFFFFu) != 0);
      const uint32_t bh = __ballot_sync(0xffffffffu, (any >> 16) != 0);
      if (lane == 0) sh.bitmap[warp] = uint16_t(bl), sh.bitmap[32 + warp] = uint16_t(bh);
    }
    __syncthreads();
    if (warp == 0) {  // the largest logit: the first bin of the first segment
      const SegmentList mine(list_word(sh.bitmap, lane), lane);
      uint32_t top = 0;
      if (mine.n > 0) {
        const Row<1> one{sh, lane, INFINITY, f.slope, 0, false};  // weights are not used
        const typename Row<1>::Bins b = one.bins(mine.at(0, lane));
        const int src = __ffs(__ballot_sync(0xffffffffu, (b.c1 | b.c0) != 0)) - 1;
        top = 1 + __shfl_sync(0xffffffffu, b.c1 ? b.bits1 : b.bits0, src);
      }
      if (lane == 0) sh.top = top;
    }
    sync_cluster<C>();

    uint32_t live = 0, top = 0, moved = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      live |= list_word(C == 1 ? sh.bitmap : peer(sh.bitmap, r), lane);
      const uint32_t t = *(C == 1 ? &sh.top : peer(&sh.top, r));
      moved |= *(C == 1 ? &sh.spills : peer(&sh.spills, r));
      if (t != 0 && (top == 0 || order_of(t - 1) > order_of(top - 1))) top = t;
    }
    const bool empty = top == 0;  // no logit above -inf
    Row<C> s{sh, lane, value_of(top - 1), f.slope, 0, moved != 0};
    if (!empty) {
      float low = s.top;
      if (f.slope.hi >= 0.f && top - 1 != kInf) low = __fmaf_rn(-kWindow, values.temperature, s.top);
      const uint32_t lb = __float_as_uint(low) >> 16;  // towards 0: a negative one's own segment or one before
      const int seg = (lb & 0x8000u) ? 512 + int(min((lb & 0x7FFFu) + 1, kInf) >> 6) : 511 - int(lb >> 6);
      // segments up to that one
      const int here = seg - 32 * lane;
      live = here >= 31 ? live : (here < 0 ? 0u : live & ~(0x7FFFFFFFu >> here));
      const SegmentList list(live, lane);
      s.n = list.n;
      for (int j = int(rank) * kWarps + warp; j < list.n; j += C * kWarps) {
        const uint32_t index = list.at(j, lane);
        const typename Row<C>::Bins b = s.bins(index);
        const u64 mass = warp_sum_u64(b.c1 * b.w1 + b.c0 * b.w0);
        const uint32_t count = uint32_t(redux_add(int(b.c1 + b.c0)));
        if (lane == 0) *(C == 1 ? &sh.seg[j] : peer(&sh.seg[j], 0)) = Segment{mass, count, index};
      }
    }
    sync_cluster<C>();

    if (rank == 0 && warp == 0 && !empty) {
      u64 kept = 0;
      uint32_t count = 0;
      for (int i0 = 0; i0 < s.n; i0 += 32) {
        const int j = i0 + lane;
        const Segment e = j < s.n ? sh.seg[j] : Segment{0, 0, 0};
        const u64 cm = warp_scan(e.mass);
        const uint32_t cc = warp_scan(e.count);
        if (j < s.n) sh.mass_before[j] = kept + cm - e.mass, sh.count_before[j] = count + cc - e.count;
        kept += __shfl_sync(0xffffffffu, cm, 31);
        count += __shfl_sync(0xffffffffu, cc, 31);
      }
      __syncwarp();
      Place last{};  // the last place that stays, unless all do
      bool whole = true;
      if (f.top_k < g.V && uint32_t(f.top_k) <= count) {  // beyond `count` tokens have no weight
        last = s.find(true, f.top_k - 1);
        kept = last.before + (last.rank + 1) * last.weight;
        whole = false;
      }
      if (f.top_p <= 1.f) {
        const u64 limit = max(mass_limit(f.top_p, kept), u64(1));
        last = s.find(false, min(limit, kept) - 1);
        kept = last.before + (last.rank + 1) * last.weight;
        whole = false;
      }
      if (f.min_w > 0 && (whole || last.weight < f.min_w)) kept = s.mass_from(f.min_w);
      const Place at = s.find(false, mass_target(f.u, kept));
      // which CTA's chunk has it
      uint32_t left = uint32_t(at.rank), owner = 0;
#pragma unroll
      for (int r = 0; r + 1 < C; ++r) {
        const uint32_t v = *peer(&sh.hist[at.bits & 0x7FFFu], r);
        uint32_t n = (at.bits & 0x8000u) ? v >> 16 : v & 0xFFFFu;
        if (s.spills)
          for (uint32_t i = 0; i < *peer(&sh.spills, r); ++i)
            n += peer(&sh.spill[i], r)->bits == at.bits ? peer(&sh.spill[i], r)->count : 0;
        if (owner == uint32_t(r) && left >= n) left -= n, ++owner;
      }
      if (lane < C) {
        *(C == 1 ? &sh.pick_bits : peer(&sh.pick_bits, lane)) = at.bits;
        *(C == 1 ? &sh.pick_rank : peer(&sh.pick_rank, lane)) = left;
        *(C == 1 ? &sh.pick_owner : peer(&sh.pick_owner, lane)) = owner;
        *(C == 1 ? &sh.kept : peer(&sh.kept, lane)) = kept;
      }
    }
    if (warp != 0 && pick_row >= 0) look_up(g, sh, pick_row, int(rank));  // of the row before this one
    sync_cluster<C>();

    pick_row = -1;
    if (empty) {
      if (rank == 0 && threadIdx.x == 0) {
        g.token[m] = -1;
        if (g.prob) g.prob[m] = 0.f;
      }
    } else if (rank == sh.pick_owner) {
      pick_row = m;
      if (threadIdx.x == 0) sh.pick = Pick{sh.pick_bits, sh.pick_rank, sh.kept, s.top, f.slope};
    }
    // clear what was hit (both signs share the words): warp w its 16 segments
    for (uint32_t bits = sh.bitmap[warp] | sh.bitmap[32 + warp]; bits; bits &= bits - 1)
      reinterpret_cast<uint2*>(sh.hist)[(warp * 16 + __ffs(bits) - 1) * 32 + lane] = make_uint2(0, 0);
    if (threadIdx.x == 0) sh.spills = 0;
    __syncthreads();  // the cleared histogram, before the next row's
  }
  if (warp != 0 && pick_row >= 0) look_up(g, sh, pick_row, int(rank));
  pdl_launch_dependents();
}

template <int C>
cudaError_t launch_rows(const Args& g, cudaStream_t s) {
  const int64_t clusters = std::min<int64_t>(g.M, clusters_at_once(C));
  return launch_clusters<C>(sample_bf16_kernel<C>, clusters * C, kThreads, int(sizeof(Shared)), s, g);
}

}  // namespace

cudaError_t launch_sample_bf16(const SampleArgs& args, cudaStream_t s) {
  // Measured per row and CTA: 8 us beside the histogram, 0.08 ns per logit.
  const int c = ctas_per_row(args.M, [&](int c) { return 8000.0 + 0.08 * double(args.V) / c; });
  SampleArgs g = args;
  g.chunk = int(((g.V + 7 + c - 1) / c + 7) / 8 * 8);
  switch (c) {
    case 1: return launch_rows<1>(g, s);
    case 2: return launch_rows<2>(g, s);
    case 4: return launch_rows<4>(g, s);
    default: return launch_rows<8>(g, s);
  }
}

}  // namespace bl
