// Sampling from bf16 logits (bl_sample).  A row has at most 65281 different
// live values, so a histogram over the 16-bit keys says everything: one
// weight per different value times an exact count, and the order of the
// tokens is the order of the bins.  No exp per logit, one shared-memory
// atomic per logit.
//
// A cluster of C CTAs takes a row, each CTA a chunk of at most 65528 logits,
// so that the 65536 counters fit in 16 bits each (128 KB): no counter can
// overflow.  Then each CTA owns a slice of the bins (read from all C
// histograms through distributed shared memory), every thread a few units of
// 8 bins in falling order, and a place in the order is found by a scan over
// the threads: the thread in whose bins a cumulative count or weight passes
// the goal knows the place.
#include "bl_internal.h"
#include "sample_weight.cuh"

namespace bl {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kUnits = 65536 / 8;            // units of 8 keys, 16 bytes of counters each
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

struct Place {
  uint32_t key, pad;
  u64 rank, before, weight;
};

struct Shared {
  uint4 hist[kUnits];
  Exp2Table exp2;
  u64 warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  uint32_t warp_max[kWarps];
  // read by the other CTAs of the cluster
  uint32_t top, local[2];
  u64 total_mass, total_count, min_mass;
  Place place[3];
  uint32_t pick[kWarps];
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

template <int C>
__device__ __forceinline__ void sync_cluster() {
  if (C == 1)
    __syncthreads();
  else
    cluster_sync();
}

template <int C>
struct Sampler {
  Shared& sh;
  const uint32_t rank;
  float top;
  Slope slope;
  int first_unit, units, per;  // falling units of the window; units of a thread
  uint32_t count;              // of this thread's bins, of those before them
  u64 mass, mass_before;
  u64 count_before;

  // Counters of a unit over the whole row.
  __device__ __forceinline__ void unit_counts(int unit, uint32_t (&c)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const uint4 q = *(C == 1 ? &sh.hist[unit] : peer(&sh.hist[unit], r));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[2 * j] += w[j] & 0xFFFFu;
        c[2 * j + 1] += w[j] >> 16;
      }
    }
  }
  __device__ __forceinline__ u64 weight(uint32_t key) const { return weight_of(value_of(key), top, slope, sh.exp2); }

  // Count and weight of this thread's bins, and of all before them.
  __device__ __forceinline__ void scan() {
    count = 0;
    mass = 0;
    const int d0 = (int(rank) * kThreads + int(threadIdx.x)) * per;
    for (int i = 0; i < per && d0 + i < units; ++i) {
      uint32_t c[8];
      const int unit = first_unit - (d0 + i);
      unit_counts(unit, c);
#pragma unroll 1
      for (int j = 7; j >= 0; --j) {
        uint32_t n = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) n = e == j ? c[e] : n;
        if (n) {
          count += n;
          mass += n * weight(unit * 8 + j);
        }
      }
    }
    uint32_t cs = count;
    u64 ms = mass;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t c = __shfl_up_sync(0xffffffffu, cs, o);
      const u64 m = __shfl_up_sync(0xffffffffu, ms, o);
      if (lane >= o) cs += c, ms += m;
    }
    if (lane == 31) sh.warp_count[warp] = cs, sh.warp_mass[warp] = ms;
    __syncthreads();
    u64 cb = 0, mb = 0, ct = 0, mt = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) cb = ct, mb = mt;
      ct += sh.warp_count[w];
      mt += sh.warp_mass[w];
    }
    if (threadIdx.x == 0) sh.total_count = ct, sh.total_mass = mt;
    sync_cluster<C>();
    if (C > 1)
      for (uint32_t r = 0; r < rank; ++r) cb += *peer(&sh.total_count, r), mb += *peer(&sh.total_mass, r);
    count_before = cb + cs - count;
    mass_before = mb + ms - mass;
  }

  __device__ __forceinline__ u64 total_mass() const {
    u64 t = 0;
    for (uint32_t r = 0; r < C; ++r) t += C == 1 ? sh.total_mass : *peer(&sh.total_mass, r);
    return t;
  }

  // The place where the cumulative count or weight first exceeds `goal`; the
  // one thread that finds it tells all CTAs through slot `slot`.
  __device__ __forceinline__ Place find(bool by_count, u64 goal, int slot) {
    const u64 at = by_count ? count_before : mass_before;
    const u64 mine = by_count ? count : mass;
    if (at <= goal && goal - at < mine) {
      u64 cb = count_before, mb = mass_before;
      const int d0 = (int(rank) * kThreads + int(threadIdx.x)) * per;
      bool done = false;
      for (int i = 0; i < per && d0 + i < units && !done; ++i) {
        uint32_t c[8];
        const int unit = first_unit - (d0 + i);
        unit_counts(unit, c);
#pragma unroll 1
        for (int j = 7; j >= 0 && !done; --j) {
          uint32_t n = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) n = e == j ? c[e] : n;
          if (!n) continue;
          const u64 w = weight(unit * 8 + j);
          if (by_count ? goal - cb < n : goal - mb < n * w) {
            const Place p{uint32_t(unit * 8 + j), 0u, by_count ? goal - cb : (goal - mb) / w, mb, w};
            for (uint32_t r = 0; r < C; ++r) *(C == 1 ? &sh.place[slot] : peer(&sh.place[slot], r)) = p;
            done = true;
          }
          cb += n;
          mb += n * w;
        }
      }
    }
    sync_cluster<C>();
    return sh.place[slot];
  }

  // Weight of the bins whose weight is at least `min_w`.
  __device__ __forceinline__ u64 mass_from(u64 min_w) {
    u64 m = 0;
    const int d0 = (int(rank) * kThreads + int(threadIdx.x)) * per;
    for (int i = 0; i < per && d0 + i < units && mass > 0; ++i) {
      uint32_t c[8];
      const int unit = first_unit - (d0 + i);
      unit_counts(unit, c);
#pragma unroll 1
      for (int j = 7; j >= 0; --j) {
        uint32_t n = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) n = e == j ? c[e] : n;
        const u64 w = n ? weight(unit * 8 + j) : 0;
        if (w >= min_w) m += n * w;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if ((threadIdx.x & 31) == 0) sh.warp_mass[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0;
    for (int w = 0; w < kWarps; ++w) m += sh.warp_mass[w];
    if (C == 1) return m;
    if (threadIdx.x == 0) sh.min_mass = m;
    cluster_sync();
    m = 0;
    for (uint32_t r = 0; r < C; ++r) m += *peer(&sh.min_mass, r);
    return m;
  }
};

template <int C>
__global__ void __launch_bounds__(kThreads) sample_bf16_kernel(const Args g) {
  extern __shared__ uint4 smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const uint32_t rank = C == 1 ? 0 : cluster_ctarank();
  const int64_t m = blockIdx.x / C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kUnits; i += kThreads) sh.hist[i] = make_uint4(0, 0, 0, 0);
  fill_exp2_table(sh.exp2);
  if (threadIdx.x < 2) sh.local[threadIdx.x] = 0;
  pdl_wait();
  __syncthreads();

  // the chunk's histogram
  const uint16_t* row = g.logits + m * g.V;
  const int off = int((reinterpret_cast<uintptr_t>(row) >> 1) & 7);
  const uint16_t* row16 = row - off;
  const int64_t end = off + g.V;
  const int64_t g0 = int64_t(rank) * (g.chunk / 8);
  const int64_t g1 = min(g0 + g.chunk / 8, (end + 7) / 8);
  uint32_t* words = reinterpret_cast<uint32_t*>(sh.hist);
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
  if (warp == 0) {
    hi = redux_max_u32(sh.warp_max[lane]);
    if (lane == 0) {
      sh.top = hi == kZeroKey - 1 ? kZeroKey : hi;
      // -0 counts as 0
      const uint32_t n = words[(kZeroKey - 1) >> 1] >> 16;
      words[(kZeroKey - 1) >> 1] &= 0xFFFFu;
      words[kZeroKey >> 1] += n;
    }
  }
  sync_cluster<C>();
  hi = sh.top;
  if (C > 1) {
    hi = 0;
    for (uint32_t r = 0; r < C; ++r) hi = max(hi, *peer(&sh.top, r));
  }
  if (hi == 0) {  // no live logit; the same in every CTA
    if (rank == 0 && threadIdx.x == 0) {
      g.token[m] = -1;
      if (g.prob) g.prob[m] = 0.f;
    }
    if (C > 1) cluster_sync();
    pdl_launch_dependents();
    return;
  }

  const RowFilter f = row_filter(m, g.V, g.temperature, g.top_k, g.top_p, g.min_p, g.u);
  const float top = value_of(hi);
  uint32_t lo = hi;
  if (f.slope.hi >= 0.f && hi < kHighKey) {
    const float t = g.temperature ? g.temperature[m] : 1.f;
    lo = max(kLowKey, key_of_f32(__fmaf_rn(-kWindow, t, top)) >> 16);
  }
  Sampler<C> s{sh, rank, top, f.slope};
  s.first_unit = hi >> 3;
  s.units = int(hi >> 3) - int(lo >> 3) + 1;
  s.per = (s.units + C * kThreads - 1) / (C * kThreads);
  s.scan();

  Place endp{0, 0, 0, 0, 0};
  u64 kept = s.total_mass();
  bool whole = true;
  if (f.top_k < g.V) {
    u64 n = 0;
    for (uint32_t r = 0; r < C; ++r) n += C == 1 ? sh.total_count : *peer(&sh.total_count, r);
    if (u64(f.top_k) <= n) {  // otherwise the k-th token has no weight
      endp = s.find(true, f.top_k - 1, 0);
      kept = endp.before + (endp.rank + 1) * endp.weight;
      whole = false;
    }
  }
  if (f.top_p <= 1.f) {
    const u64 limit = max(mass_limit(f.top_p, kept), u64(1));
    endp = s.find(false, min(limit, kept) - 1, 1);
    kept = endp.before + (endp.rank + 1) * endp.weight;
    whole = false;
  }
  if (f.min_w > 0 && (whole || endp.weight < f.min_w)) kept = s.mass_from(f.min_w);
  const Place at = s.find(false, mass_target(f.u, kept), 2);

  // the element of that key with at.rank equal ones before it, in index order
  auto local_count = [&](uint32_t r) {
    const uint32_t w = *(C == 1 ? &words[at.key >> 1] : peer(&words[at.key >> 1], r));
    return (w >> (16 * (at.key & 1))) & 0xFFFFu;
  };
  u64 want = at.rank;
  uint32_t owner = 0;
  if (C > 1)
    for (; owner + 1 < C; ++owner) {
      const uint32_t n = local_count(owner);
      if (want < n) break;
      want -= n;
    }
  if (C > 1) cluster_sync();  // the last read of another CTA's memory
  if (rank == owner) {
    // warps take contiguous ranges of groups; a warp counts, then the one that has the element walks
    const int64_t n = g1 - g0, span = (n + kWarps - 1) / kWarps;
    const int64_t w0 = g0 + warp * span, w1 = min(w0 + span, g1);
    auto match = [&](int64_t i) {
      uint32_t k[4], b = 0;
      load_keys(row16, off, end, i, k);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t key = (k[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
        key += key == kZeroKey - 1;
        b |= uint32_t(key == at.key) << j;
      }
      return b;
    };
    uint32_t mine = 0;
    for (int64_t i = w0 + lane; i < w1; i += 32) mine += __popc(match(i));
    mine = redux_add(int(mine));
    if (lane == 0) sh.pick[warp] = mine;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += sh.pick[w];
    if (before <= want && want - before < mine) {
      uint32_t left = uint32_t(want) - before;
      for (int64_t i0 = w0; i0 < w1; i0 += 32) {
        const uint32_t b = i0 + lane < w1 ? match(i0 + lane) : 0;
        uint32_t incl = __popc(b);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
        const uint32_t excl = incl - __popc(b);
        if (left < all && left >= excl && left < incl) {
          uint32_t bits = b;
          for (uint32_t q = left - excl; q > 0; --q) bits &= bits - 1;
          g.token[m] = int32_t((i0 + lane) * 8 + (__ffs(bits) - 1) - off);
          if (g.prob) g.prob[m] = share_of(value_of(at.key), top, f.slope, sh.exp2, kept);
        }
        if (left < all) break;
        left -= all;
      }
    }
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
  cfg.gridDim = dim3(unsigned(g.M * C));
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
  if (chunk_of(c) > kMaxChunk || M * c > 0x7fffffff) return cudaErrorNotSupported;
  const Args g{logits, temperature, top_p, min_p, u, top_k, M, V, token, prob, int(chunk_of(c))};
  switch (c) {
    case 1: return launch_rows<1>(g, s);
    case 2: return launch_rows<2>(g, s);
    case 4: return launch_rows<4>(g, s);
    default: return launch_rows<8>(g, s);
  }
}

}  // namespace bl
