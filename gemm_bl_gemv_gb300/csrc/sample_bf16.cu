// Sampling from bf16 logits (bl_sample).  A row has at most 65281 different
// live values, so a histogram over the 16-bit keys says everything: one
// weight per different value times an exact count, and the order of the
// tokens is the order of the bins.  No exp per logit, one shared-memory
// atomic per logit.
//
// A cluster of C CTAs takes a row, each CTA a chunk of at most 65528 logits,
// so that the 65536 counters fit in 16 bits each (128 KB): no counter can
// overflow.  The bins are cut into 1024 segments of 64; only the segments
// that some CTA has hit (some tens, of a model's logits) are weighed, one
// warp each, with the counts of all C histograms read through distributed
// shared memory.  One warp of the first CTA then finds the places in the
// order: first the segment in which a cumulative count or weight passes the
// goal, then the bin.  The CTA whose chunk has the token looks up its index.
// Clusters stay for several rows and clear only the segments that they hit.
#include "bl_internal.h"
#include "sample_weight.cuh"

namespace bl {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kUnits = 65536 / 8;            // units of 8 keys, 16 bytes of counters each
constexpr int kSegments = 65536 / 64;        // segments of 64 keys, 32 words of counters
constexpr int kMaxChunk = 65528;             // logits of a CTA: a counter stays below 2^16
constexpr uint32_t kLowKey = 0x0080u;        // the lowest finite value; -inf and NaN lie below
constexpr uint32_t kHighKey = 0xFF80u;       // +inf; NaN above
constexpr uint32_t kZeroKey = 0x8000u;       // 0; 0x7fff is -0
// weights below 2^-45 of the largest are 0: no bin further than 46 octaves (31.9 T) matters
constexpr float kWindow = 32.f;

struct Args {
  const uint16_t* logits;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int64_t M, V;
  int32_t* token;
  float* prob;
  int chunk;  // a multiple of 8
};

// A place in the order: the element of this key with `rank` others of the
// same key before it; `before` is the weight of everything before that key.
struct Place {
  uint32_t key;
  u64 rank, before, weight;
};

struct Segment {
  u64 mass;
  uint32_t count, index;
};

struct Shared {
  uint4 hist[kUnits];
  // read by the other CTAs of the cluster
  uint32_t bitmap[32];  // segments that this CTA has hit
  uint32_t top;         // its largest key, 0 if it has no live logit
  // written by the other CTAs (to rank 0's), in falling order
  Segment seg[kSegments];
  // written by rank 0
  uint32_t pick_key, pick_rank, pick_owner;
  u64 kept;
  // local
  u64 mass_before[kSegments];
  uint32_t count_before[kSegments];
  Exp2Table exp2;
  uint32_t warp_max[kWarps], pick[kWarps];
};

template <class T>
__device__ __forceinline__ T* peer(T* p, uint32_t rank) {
  uint64_t a;
  asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(a);
}

// Keys of two packed bf16 values.
__device__ __forceinline__ uint32_t keys2(uint32_t w) {
  const uint32_t s = (w >> 15) & 0x00010001u;
  return w ^ (((s << 15) - s) | 0x80008000u);
}
__device__ __forceinline__ float value_of(uint32_t key) { return f32_of_key(key << 16 | ((key & 0x8000u) ? 0u : 0xFFFFu)); }

// The 8 logits of group `grp` (aligned in memory) as keys; those outside the
// row are 0, a NaN's key.  `row16` is the 16-byte aligned start, `off` the
// row's first element in it.
__device__ __forceinline__ void load_keys(const uint16_t* row16, int off, int64_t end, int64_t grp, uint32_t (&k)[4]) {
  const int64_t v = grp * 8;
  if (v >= off && v + 8 <= end) {
    const uint4 q = reinterpret_cast<const uint4*>(row16)[grp];
    k[0] = keys2(q.x);
    k[1] = keys2(q.y);
    k[2] = keys2(q.z);
    k[3] = keys2(q.w);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w = 0;
    const int64_t i = v + 2 * j;
    if (i >= off && i < end) w = row16[i];
    uint32_t key = keys2(w) & 0xFFFFu;
    if (i < off || i >= end) key = 0;
    w = 0;
    if (i + 1 >= off && i + 1 < end) w = row16[i + 1];
    uint32_t key1 = keys2(w) & 0xFFFFu;
    if (i + 1 < off || i + 1 >= end) key1 = 0;
    k[j] = key | key1 << 16;
  }
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int C>
__device__ __forceinline__ void sync_cluster() {
  if (C == 1)
    __syncthreads();
  else
    cluster_sync();
}

// The live segments of a row in falling order, held by a warp: lane i has the
// bits of word 31 - i, highest first.
struct SegmentList {
  uint32_t bits, upto;  // segments of this lane and the lanes before it
  int n;
  __device__ __forceinline__ SegmentList(uint32_t word, int lane) {
    bits = word;
    upto = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
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
    return 32u * (31 - src) + 31 - (__ffs(__ballot_sync(0xffffffffu, here)) - 1);
  }
};

template <int C>
struct Row {
  Shared& sh;
  int lane;
  float top;
  Slope slope;
  int n;  // live segments

  __device__ __forceinline__ u64 weight(uint32_t key) const { return weight_of(value_of(key), top, slope, sh.exp2); }

  // This lane's two bins of a segment, in falling order: keys k and k - 1.
  struct Bins {
    uint32_t key, c1, c0;
    u64 w1, w0;
  };
  __device__ __forceinline__ Bins bins(uint32_t seg) const {
    Bins b;
    const uint32_t word = seg * 32 + 31 - lane;
    b.key = 2 * word + 1;
    b.c1 = b.c0 = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const uint32_t* mine = reinterpret_cast<uint32_t*>(sh.hist) + word;
      const uint32_t v = *(C == 1 ? mine : peer(mine, r));
      b.c1 += v >> 16;
      b.c0 += v & 0xFFFFu;
    }
    b.w1 = b.c1 ? weight(b.key) : 0;
    b.w0 = b.c0 ? weight(b.key - 1) : 0;
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
      u64 cm = m1 + m0;
      uint32_t cc = b.c1 + b.c0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 m = __shfl_up_sync(0xffffffffu, cm, o);
        const uint32_t c = __shfl_up_sync(0xffffffffu, cc, o);
        if (lane >= o) cm += m, cc += c;
      }
      const u64 before = sh.mass_before[s] + cm - m1 - m0;
      const u64 at = by_count ? u64(sh.count_before[s]) + cc - b.c1 - b.c0 : before;
      const u64 n1 = by_count ? b.c1 : m1, n0 = by_count ? b.c0 : m0;
      const bool in1 = at <= goal && goal - at < n1;
      const bool in0 = at + n1 <= goal && goal - at - n1 < n0;
      Place p{};
      if (in1) p = Place{b.key, by_count ? goal - at : (goal - at) / b.w1, before, b.w1};
      if (in0) p = Place{b.key - 1, by_count ? goal - at - n1 : (goal - at - n1) / b.w0, before + m1, b.w0};
      const int src = __ffs(__ballot_sync(0xffffffffu, in1 || in0)) - 1;
      p.key = __shfl_sync(0xffffffffu, p.key, src);
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
      const bool less = i < n && weight(max(sh.seg[i].index * 64, kLowKey)) < min_w;
      const uint32_t hit = __ballot_sync(0xffffffffu, less);
      if (!hit) continue;
      const int s = i0 + __ffs(hit) - 1;
      const Bins b = bins(sh.seg[s].index);
      return sh.mass_before[s] + warp_sum_u64((b.w1 >= min_w ? b.c1 * b.w1 : 0) + (b.w0 >= min_w ? b.c0 * b.w0 : 0));
    }
    return sh.mass_before[n - 1] + sh.seg[n - 1].mass;
  }
};

template <int C>
__global__ void __launch_bounds__(kThreads) sample_bf16_kernel(const Args g) {
  extern __shared__ uint4 smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const uint32_t rank = C == 1 ? 0 : cluster_ctarank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* words = reinterpret_cast<uint32_t*>(sh.hist);
  for (int i = threadIdx.x; i < kUnits; i += kThreads) sh.hist[i] = make_uint4(0, 0, 0, 0);
  fill_exp2_table(sh.exp2);
  pdl_wait();
  __syncthreads();

  for (int64_t m = blockIdx.x / C; m < g.M; m += gridDim.x / C) {
    const RowFilter f = row_filter(m, g.V, g.temperature, g.top_k, g.top_p, g.min_p, g.u);
    const float temp = g.temperature ? g.temperature[m] : 1.f;

    // the chunk's histogram
    const uint16_t* row = g.logits + m * g.V;
    const int off = int((reinterpret_cast<uintptr_t>(row) >> 1) & 7);
    const uint16_t* row16 = row - off;
    const int64_t end = off + g.V;
    const int64_t g0 = int64_t(rank) * (g.chunk / 8);
    const int64_t g1 = min(g0 + g.chunk / 8, (end + 7) / 8);
    uint32_t hi = 0;
    for (int64_t i = g0 + threadIdx.x; i < g1; i += kThreads) {
      uint32_t k[4];
      load_keys(row16, off, end, i, k);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t key = (k[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
        if (key - kLowKey <= kHighKey - kLowKey) {
          hi = max(hi, key);
          atomicAdd(&words[key >> 1], 1u << (16 * (key & 1)));
        }
      }
    }
    hi = redux_max_u32(hi);
    if (lane == 0) sh.warp_max[warp] = hi;
    __syncthreads();
    if (threadIdx.x == 0) {  // -0 counts as 0
      const uint32_t neg = words[(kZeroKey - 1) >> 1] >> 16;
      words[(kZeroKey - 1) >> 1] &= 0xFFFFu;
      words[kZeroKey >> 1] += neg;
    }
    __syncthreads();
    // which segments were hit: a warp reads four (512 bytes) at a time
    for (int w = warp; w < 32; w += kWarps) {
      uint32_t bits = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint4 v = sh.hist[(w * 8 + q) * 32 + lane];
        const uint32_t b = __ballot_sync(0xffffffffu, (v.x | v.y | v.z | v.w) != 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) bits |= uint32_t(((b >> (8 * e)) & 0xFFu) != 0) << (4 * q + e);
      }
      if (lane == 0) sh.bitmap[w] = bits;
    }
    if (warp == 0) {
      hi = redux_max_u32(sh.warp_max[lane]);
      if (lane == 0) sh.top = hi == kZeroKey - 1 ? kZeroKey : hi;
    }
    sync_cluster<C>();

    uint32_t live = 0;  // lane i: word 31 - i of all CTAs' bitmaps
    hi = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      live |= *(C == 1 ? &sh.bitmap[31 - lane] : peer(&sh.bitmap[31 - lane], r));
      hi = max(hi, *(C == 1 ? &sh.top : peer(&sh.top, r)));
    }
    Row<C> s{sh, lane, value_of(hi), f.slope, 0};
    if (hi != 0) {
      uint32_t lo = hi;
      if (f.slope.hi >= 0.f && hi < kHighKey) lo = max(kLowKey, key_of_f32(__fmaf_rn(-kWindow, temp, s.top)) >> 16);
      // segments from lo's on
      const int from = int(lo >> 6) - 32 * (31 - lane);
      live = from <= 0 ? live : (from < 32 ? live & (0xFFFFFFFFu << from) : 0u);
      const SegmentList list(live, lane);
      s.n = list.n;
      for (int i = int(rank) * kWarps + warp; i < list.n; i += C * kWarps) {
        const uint32_t seg = list.at(i, lane);
        const typename Row<C>::Bins b = s.bins(seg);
        const u64 mass = warp_sum_u64(b.c1 * b.w1 + b.c0 * b.w0);
        const uint32_t count = uint32_t(redux_add(int(b.c1 + b.c0)));
        if (lane == 0) *(C == 1 ? &sh.seg[i] : peer(&sh.seg[i], 0)) = Segment{mass, count, seg};
      }
    }
    sync_cluster<C>();

    if (rank == 0 && warp == 0 && hi != 0) {
      u64 kept = 0;
      uint32_t count = 0;
      for (int i0 = 0; i0 < s.n; i0 += 32) {
        const int i = i0 + lane;
        const Segment e = i < s.n ? sh.seg[i] : Segment{0, 0, 0};
        u64 cm = e.mass;
        uint32_t cc = e.count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 v = __shfl_up_sync(0xffffffffu, cm, o);
          const uint32_t c = __shfl_up_sync(0xffffffffu, cc, o);
          if (lane >= o) cm += v, cc += c;
        }
        if (i < s.n) sh.mass_before[i] = kept + cm - e.mass, sh.count_before[i] = count + cc - e.count;
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
        const uint32_t v = *peer(&words[at.key >> 1], r);
        const uint32_t c = (v >> (16 * (at.key & 1))) & 0xFFFFu;
        if (owner == uint32_t(r) && left >= c) left -= c, ++owner;
      }
      if (lane < C) {
        *(C == 1 ? &sh.pick_key : peer(&sh.pick_key, lane)) = at.key;
        *(C == 1 ? &sh.pick_rank : peer(&sh.pick_rank, lane)) = left;
        *(C == 1 ? &sh.pick_owner : peer(&sh.pick_owner, lane)) = owner;
        *(C == 1 ? &sh.kept : peer(&sh.kept, lane)) = kept;
      }
    }
    sync_cluster<C>();

    // clear what was hit: warp w the segments of word w
    for (int w = warp; w < 32; w += kWarps)
      for (uint32_t bits = sh.bitmap[w]; bits; bits &= bits - 1) words[(w * 32 + __ffs(bits) - 1) * 32 + lane] = 0;

    if (hi == 0) {
      if (rank == 0 && threadIdx.x == 0) {
        g.token[m] = -1;
        if (g.prob) g.prob[m] = 0.f;
      }
    } else if (rank == sh.pick_owner) {
      // the element of that key with `want` equal ones before it in the chunk: warps take contiguous
      // ranges of groups and keep the matches of each, at most kMaxChunk / 8 / kWarps / 32 = 8 per lane
      const uint32_t key_at = sh.pick_key, want = sh.pick_rank;
      const int n = int(g1 - g0), span = (n + kWarps - 1) / kWarps;
      const int64_t w0 = g0 + warp * span;
      const int wn = max(0, min(span, n - warp * span));
      u64 found = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (q * 32 + lane < wn) {
          uint32_t k[4], b = 0;
          load_keys(row16, off, end, w0 + q * 32 + lane, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t key = (k[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
            key += key == kZeroKey - 1;
            b |= uint32_t(key == key_at) << j;
          }
          found |= u64(b) << (8 * q);
        }
      }
      const uint32_t mine = uint32_t(redux_add(__popcll(found)));
      if (lane == 0) sh.pick[warp] = mine;
      __syncthreads();
      const uint32_t before = uint32_t(redux_add(lane < warp ? int(sh.pick[lane]) : 0));
      if (before <= want && want - before < mine) {
        uint32_t left = want - before;
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          const uint32_t b = uint32_t(found >> (8 * q)) & 0xFFu;
          const uint32_t all = uint32_t(redux_add(__popc(b)));
          if (left >= all) {
            left -= all;
            continue;
          }
          uint32_t excl = __popc(b);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, excl, o);
            if (lane >= o) excl += v;
          }
          excl -= __popc(b);
          if (left >= excl && left - excl < uint32_t(__popc(b))) {
            uint32_t bits = b;
            for (uint32_t e = left - excl; e > 0; --e) bits &= bits - 1;
            g.token[m] = int32_t((w0 + q * 32 + lane) * 8 + (__ffs(bits) - 1) - off);
            if (g.prob) g.prob[m] = share_of(value_of(key_at), s.top, f.slope, sh.exp2, sh.kept);
          }
          break;
        }
      }
    }
    __syncthreads();  // the cleared histogram, before the next row's
  }
  pdl_launch_dependents();
}

template <int C>
cudaError_t launch_rows(const Args& g, cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = raise_smem_cap(sample_bf16_kernel<C>, dev, int(sizeof(Shared)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(g.M, std::max(1, sm_count() / C)) * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (C > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim = {C, 1, 1};
    ++n;
  }
  if (overlap_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, sample_bf16_kernel<C>, g);
}

}  // namespace

// cudaErrorNotSupported, having launched nothing, for rows too long for eight chunks.
cudaError_t launch_sample_bf16(const uint16_t* logits, const float* temperature, const int32_t* top_k,
                               const float* top_p, const float* min_p, const float* u, int64_t M, int64_t V,
                               int32_t* token, float* prob, cudaStream_t s) {
  auto chunk_of = [&](int c) { return ((V + 7 + c - 1) / c + 7) / 8 * 8; };
  int c = 1;
  while (c < 8 && (chunk_of(c) > kMaxChunk || (M * c * 2 <= sm_count() && chunk_of(c) > 8 * kThreads))) c *= 2;
  if (chunk_of(c) > kMaxChunk) return cudaErrorNotSupported;
  const Args g{logits, temperature, top_p, min_p, u, top_k, M, V, token, prob, int(chunk_of(c))};
  switch (c) {
    case 1: return launch_rows<1>(g, s);
    case 2: return launch_rows<2>(g, s);
    case 4: return launch_rows<4>(g, s);
    default: return launch_rows<8>(g, s);
  }
}

}  // namespace bl
