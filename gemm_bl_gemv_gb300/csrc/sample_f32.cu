// Sampling from fp32 logits (bl_sample).  A cluster of C CTAs takes a row.
// The order of the tokens is found by a radix descent whose first digit is
// linear in the exponent z = (max - l) log2(e) / T: 2048 bins over the octaves
// that have weight (46, or the row's range), so a bin holds values whose
// weights differ by at most 1.6 %.  One pass counts the logits of every bin
// and sums their weights, as 31-bit integers relative to a power of two of the
// bin, in two 32-bit halves: sums are exact, and atomics may add them in any
// order.  A place in the order is then found by a scan over the bins, and
// within its bin by sorting the bin's logits; a bin with more than 1024 of
// them is cut again, by the rest of z and then by the bits of the value.
//
// The first pass, for the largest logit, leaves the chunk in shared memory where
// it fits there (37000 logits), and the later passes read it from there.
//
// Bound: instruction issue in the pass that counts and weighs (some 70
// instructions per logit, 40 of them the weight: 11 us for 25001 logits a CTA;
// one atomic less, additions in place of the conversions, and a table without
// bank conflicts each changed nothing), and 7 us of exchanges in the cluster
// for every place that is looked for.  32 rows of 100003, mixed filters: 46 us.
#include "sample_common.cuh"

namespace bl {
namespace {

using Args = SampleArgs;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxChunk = 65536;  // logits of a CTA: 16-bit halves of weights add up in 32 bits
constexpr size_t kMaxShared = 227 * 1024;
constexpr float kOctaves = 46.f;  // weights below 2^-45 of the largest are 0

// A digit of the descent: counts and weights of 2048 bins.
struct Digit {
  uint32_t count[kBins], hi[kBins], lo[kBins];
};

// Over all CTAs, on rank 0: before each bin, in units of the digit.
struct Sums {
  u64 mass[kBins + 1];
  uint32_t count[kBins + 1];
};

// Where a search is: the bins that it went down to.
struct Path {
  int depth;               // digits that are fixed
  uint32_t bin[5];         // the fixed digits
  uint32_t n;              // logits of the last bin
  uint32_t before_count;   // of everything before it
  u64 before;              // weight of everything before it, in the search's unit
};

// A place in the order: a logit's key, how many equal ones come before it, its
// weight and the weight up to and with it (in units of 2^-44 of the largest).
struct Place {
  uint32_t key, rank;
  u64 weight, through;
};

struct __align__(16) Shared {
  Digit digit;
  Sums first, later;  // rank 0's: the first digit's, a later one's
  uint32_t list[kThreads];
  Exp2Table exp2;
  // exchanged in the cluster
  float high, low;
  u64 sum;
  uint32_t equal;
  uint32_t listed;
  Path path;
  Place place;
  // local
  float redf[2][kWarps];
  u64 redu[kWarps];
  uint32_t redc[kWarps];
};

template <int C>
struct Row {
  Shared& sh;
  const float* x;  // the chunk
  int n;
  uint32_t rank;
  float top;
  Slope slope;
  float scale, per_bin;  // bins per unit of max - l, octaves per bin

  template <class T>
  __device__ __forceinline__ T* at(T* p, uint32_t r) const {
    return C == 1 ? p : peer(p, r);
  }

  // f(index, logit) for this thread's logits of the chunk, eight loads at a time (a load waits for L2).
  template <class F>
  __device__ __forceinline__ void each_at(F f) const {
    int i = threadIdx.x;
    for (; i + 7 * kThreads < n; i += 8 * kThreads) {
      float l[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) l[j] = x[i + j * kThreads];
#pragma unroll
      for (int j = 0; j < 8; ++j) f(i + j * kThreads, l[j]);
    }
    float l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) l[j] = i + j * kThreads < n ? x[i + j * kThreads] : -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j * kThreads < n) f(i + j * kThreads, l[j]);
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    each_at([&](int, float l) { f(l); });
  }

  // ---- a logit's digits ----
  __device__ __forceinline__ bool live(float l) const {
    return slope.hi < 0.f ? l == top : l > -INFINITY && __fmul_rn(__fsub_rn(top, l), slope.hi) < kOctaves;
  }
  __device__ __forceinline__ float place_of(float l) const {  // rises as l falls; its whole part is the first digit
    return slope.hi < 0.f ? 0.f : fminf(__fmul_rn(__fsub_rn(top, l), scale), float(kBins) - 0.0625f);
  }
  __device__ __forceinline__ uint32_t digit_of(float l, int depth) const {
    if (depth < 2) {
      const float y = place_of(l);
      const uint32_t b = uint32_t(y);
      return depth == 0 ? b : uint32_t((y - float(b)) * float(kBins));
    }
    const uint32_t k = ~key_of_f32(l);
    return depth == 2 ? k >> 21 : depth == 3 ? (k >> 10) & 2047u : k & 1023u;
  }
  // Whether a logit is on the path; most fail the first comparison.  `from` is the path's first digit.
  __device__ __forceinline__ bool matches(float l, const Path& p, float from) const {
    if (p.depth > 0) {
      const float y = place_of(l);
      if (!(y >= from && y < from + 1.f)) return false;
    }
    if (!live(l)) return false;
    for (int d = 1; d < p.depth; ++d)
      if (digit_of(l, d) != p.bin[d]) return false;
    return true;
  }
  // The power of two that a first digit's weights are relative to, and a weight relative to it, 31 bits.
  __device__ __forceinline__ int octave_of(uint32_t bin) const { return int(float(bin) * per_bin); }
  __device__ __forceinline__ uint32_t relative(float l, int octave) const {
    int shift;
    const u64 w = weight_mantissa(l, top, slope, sh.exp2, shift);
    return uint32_t(w >> min(max(13 + shift - octave, 13), 44));
  }
  // Weight in units of 2^-44 from one relative to an octave, and back.
  __device__ __forceinline__ static u64 absolute(u64 relative, int octave) { return (relative << 13) >> octave; }
  __device__ __forceinline__ static u64 local(u64 mass, int octave) { return (mass << octave) >> 13; }

  // ---- sums over the CTA, the cluster ----
  __device__ __forceinline__ u64 cta_sum(u64 v) {
    v = warp_sum_u64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.redu[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum_u64(sh.redu[threadIdx.x & 31]);
  }
  __device__ __forceinline__ u64 cluster_total(u64 v) {
    v = cta_sum(v);
    if (C == 1) return v;
    sync_cluster<C>();  // earlier readers of sum
    if (threadIdx.x == 0) sh.sum = v;
    sync_cluster<C>();
    v = 0;
    for (uint32_t r = 0; r < C; ++r) v += *at(&sh.sum, r);
    return v;
  }

  // Count and weigh the logits on `p` by their next digit; rank 0 gets the sums before each bin.
  __device__ void cut(const Path& p, Sums& sums) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.digit.count[i] = sh.digit.hi[i] = sh.digit.lo[i] = 0;
    __syncthreads();
    const float from = p.depth > 0 ? float(p.bin[0]) : 0.f;
    each([&](float l) {
      if (!matches(l, p, from)) return;
      const uint32_t b = digit_of(l, p.depth);
      const uint32_t w = relative(l, octave_of(p.depth == 0 ? b : p.bin[0]));
      atomicAdd(&sh.digit.count[b], 1u);
      atomicAdd(&sh.digit.hi[b], w >> 16);
      atomicAdd(&sh.digit.lo[b], w & 0xFFFFu);
    });
    sync_cluster<C>();
    // each CTA adds up a slice of the bins
    constexpr int kSlice = kBins / C;
    for (int i = threadIdx.x; i < kSlice; i += kThreads) {
      const int b = int(rank) * kSlice + i;
      u64 mass = 0;
      uint32_t count = 0;
#pragma unroll
      for (uint32_t r = 0; r < C; ++r) {
        const Digit* d = at(&sh.digit, r);
        mass += (u64(d->hi[b]) << 16) + d->lo[b];
        count += d->count[b];
      }
      Sums* s = at(&sums, 0);
      s->mass[b] = p.depth == 0 ? absolute(mass, octave_of(b)) : mass;
      s->count[b] = count;
    }
    sync_cluster<C>();
    if (rank != 0) return;
    // exclusive sums, two bins per thread
    static_assert(kBins == 2 * kThreads, "");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = 2 * threadIdx.x;
    const u64 m0 = sums.mass[b], m1 = sums.mass[b + 1];
    const uint32_t c0 = sums.count[b], c1 = sums.count[b + 1];
    const u64 ms = warp_scan(m0 + m1);
    const uint32_t cs = warp_scan(c0 + c1);
    if (lane == 31) sh.redu[warp] = ms, sh.redc[warp] = cs;
    __syncthreads();
    const u64 wm = warp_sum_u64(lane < warp ? sh.redu[lane] : 0);
    const uint32_t wc = uint32_t(redux_add(lane < warp ? int(sh.redc[lane]) : 0));
    sums.mass[b] = wm + ms - m0 - m1;
    sums.mass[b + 1] = wm + ms - m1;
    sums.count[b] = wc + cs - c0 - c1;
    sums.count[b + 1] = wc + cs - c1;
    if (threadIdx.x == kThreads - 1) sums.mass[kBins] = wm + ms, sums.count[kBins] = wc + cs;
    __syncthreads();
  }

  // The bin in which the count or weight first exceeds `goal` (less than the whole), told to all CTAs.
  __device__ void descend(Path p, const Sums& sums, bool by_count, u64 goal) {
    if (rank == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = 2 * threadIdx.x + j;
        const u64 lo = by_count ? sums.count[b] : sums.mass[b], hi = by_count ? sums.count[b + 1] : sums.mass[b + 1];
        if (lo <= goal && goal < hi) {
          p.bin[p.depth] = b;
          p.n = sums.count[b + 1] - sums.count[b];
          p.before_count += sums.count[b];
          p.before += sums.mass[b];
          ++p.depth;
          for (uint32_t r = 0; r < C; ++r) *at(&sh.path, r) = p;
        }
      }
    }
    sync_cluster<C>();
  }

  // The place where the cumulative count or weight first exceeds `goal`, less than the whole.
  __device__ Place find(bool by_count, u64 goal) {
    descend(Path{}, sh.first, by_count, goal);
    Path p = sh.path;
    const int octave = octave_of(p.bin[0]);
    // within the first bin: weights relative to its octave
    const u64 outside = p.before;
    const uint32_t outside_count = p.before_count;
    goal = by_count ? goal - outside_count : local(goal - outside, octave);
    p.before = 0;
    p.before_count = 0;
    while (p.n > kThreads && p.depth < 5) {
      cut(p, sh.later);
      descend(p, sh.later, by_count, goal - (by_count ? p.before_count : p.before));
      p = sh.path;
    }
    if (p.n <= kThreads) {
      // its logits' keys, falling, one per thread of rank 0
      if (threadIdx.x == 0) sh.listed = 0;
      sync_cluster<C>();
      const float from = float(p.bin[0]);
      each([&](float l) {
        if (matches(l, p, from)) at(&sh.list[0], 0)[atomicAdd(at(&sh.listed, 0), 1u)] = key_of_f32(l);
      });
      sync_cluster<C>();
      if (rank == 0) {
        const uint32_t i = threadIdx.x;
        uint32_t key = i < p.n ? sh.list[i] : 0u;  // 0: below every logit's
        for (uint32_t k = 2; k < 2 * p.n; k <<= 1)
          for (uint32_t j = k >> 1; j > 0; j >>= 1) {
            uint32_t other;
            if (j >= 32) {
              __syncthreads();
              sh.list[i] = key;
              __syncthreads();
              other = sh.list[i ^ j];
            } else {
              other = __shfl_xor_sync(0xffffffffu, key, j);
            }
            const bool larger = ((i & k) == 0) == ((i & j) == 0);
            key = larger ? max(key, other) : min(key, other);
          }
        __syncthreads();
        sh.list[i] = key;
        const u64 w = i < p.n ? relative(f32_of_key(key), octave) : 0;
        u64 upto = warp_scan(w);
        if ((i & 31) == 31) sh.redu[i >> 5] = upto;
        __syncthreads();
        upto += p.before + warp_sum_u64((i & 31) < (i >> 5) ? sh.redu[i & 31] : 0);
        const bool here = by_count ? i + p.before_count == goal : goal >= upto - w && goal < upto;
        if (here) {
          uint32_t first = i;
          while (first > 0 && sh.list[first - 1] == key) --first;
          const Place q{key, i - first, weight_of(f32_of_key(key), top, slope, sh.exp2), outside + absolute(upto, octave)};
          for (uint32_t r = 0; r < C; ++r) *at(&sh.place, r) = q;
        }
      }
    } else if (rank == 0 && threadIdx.x == 0) {  // more than 1024 equal logits
      uint32_t key = ~(p.bin[2] << 21 | p.bin[3] << 10 | p.bin[4]);
      const u64 w = relative(f32_of_key(key), octave);
      const u64 i = by_count ? goal - p.before_count : w ? (goal - p.before) / w : 0;
      const Place q{key, uint32_t(i), weight_of(f32_of_key(key), top, slope, sh.exp2),
                    outside + absolute(p.before + (i + 1) * w, octave)};
      for (uint32_t r = 0; r < C; ++r) *at(&sh.place, r) = q;
    }
    sync_cluster<C>();
    return sh.place;
  }
};

template <int C>
__global__ void __launch_bounds__(kThreads) sample_f32_kernel(const Args g) {
  extern __shared__ uint4 smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const uint32_t rank = C == 1 ? 0 : cluster_ctarank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m = blockIdx.x / C;
  fill_exp2_table(sh.exp2);
  pdl_wait();
  const RowFilter f = row_filter(RowValues(m, g.temperature, g.top_k, g.top_p, g.min_p, g.u), g.V);
  const int begin = int(rank) * g.chunk;
  Row<C> row{sh, static_cast<const float*>(g.logits) + m * g.V + begin, max(0, min(g.chunk, int(g.V) - begin)), rank};

  // the largest and the smallest live logit
  float hi = -INFINITY, lo = INFINITY;
  float* copy = reinterpret_cast<float*>(smem + sizeof(Shared) / sizeof(uint4));
  row.each_at([&](int i, float l) {
    if (g.copy) copy[i] = l;
    hi = fmaxf(hi, l);
    if (l > -INFINITY) lo = fminf(lo, l);
  });
  hi = warp_max(hi);
  lo = -warp_max(-lo);
  if (lane == 0) sh.redf[0][warp] = hi, sh.redf[1][warp] = lo;
  __syncthreads();
  if (g.copy) row.x = copy;
  hi = warp_max(sh.redf[0][lane]);
  lo = -warp_max(-sh.redf[1][lane]);
  if (C > 1) {
    if (threadIdx.x == 0) sh.high = hi, sh.low = lo;
    sync_cluster<C>();
#pragma unroll
    for (uint32_t r = 0; r < C; ++r) hi = fmaxf(hi, *peer(&sh.high, r)), lo = fminf(lo, *peer(&sh.low, r));
  }
  if (hi == -INFINITY) {  // no live logit
    if (rank == 0 && threadIdx.x == 0) {
      g.token[m] = -1;
      if (g.prob) g.prob[m] = 0.f;
    }
    if (C > 1) sync_cluster<C>();
    pdl_launch_dependents();
    return;
  }
  row.top = hi + 0.f;
  row.slope = hi == INFINITY ? Slope{-1.f, 0.f} : f.slope;
  const float range = fminf(__fmul_rn(__fsub_rn(hi, lo), fmaxf(row.slope.hi, 0.f)), kOctaves);
  row.per_bin = range * (1.f / (kBins - 1));
  row.scale = range > 0.f ? row.slope.hi * ((kBins - 1) / range) : 0.f;
  if (!(row.scale < INFINITY)) row.scale = row.per_bin = 0.f;  // a range too small to divide by

  row.cut(Path{}, sh.first);
  sync_cluster<C>();
  u64 kept = *row.at(&sh.first.mass[kBins], 0);
  const u64 all = *row.at(&sh.first.count[kBins], 0);
  Place last{};
  bool whole = true;
  if (u64(f.top_k) < u64(g.V) && u64(f.top_k) <= all) {  // beyond them tokens have no weight
    last = row.find(true, f.top_k - 1);
    kept = last.through;
    whole = false;
  }
  if (f.top_p <= 1.f) {
    const u64 limit = max(mass_limit(f.top_p, kept), u64(1));
    last = row.find(false, min(limit, kept) - 1);
    kept = last.through;
    whole = false;
  }
  if (f.min_w > 0 && (whole || last.weight < f.min_w)) {
    kept = 0;
    row.each([&](float l) {
      const u64 w = row.live(l) ? weight_of(l, row.top, row.slope, sh.exp2) : 0;
      kept += w >= f.min_w ? w : 0;
    });
    kept = row.cluster_total(kept);
  }
  const Place p = row.find(false, mass_target(f.u, kept));

  // the logit of that key with p.rank equal ones before it: each warp counts a contiguous part of the chunk
  const int span = (row.n + kWarps - 1) / kWarps;
  const int w0 = min(row.n, warp * span), w1 = min(row.n, w0 + span);
  uint32_t mine = 0;
  for (int i = w0 + lane; i < w1; i += 32) mine += key_of_f32(row.x[i]) == p.key;
  mine = uint32_t(redux_add(int(mine)));
  __syncthreads();
  if (lane == 0) sh.redc[warp] = mine;
  __syncthreads();
  const uint32_t counts = sh.redc[lane];
  uint32_t before = uint32_t(redux_add(lane < warp ? int(counts) : 0));
  if constexpr (C > 1) {
    const uint32_t cta = uint32_t(redux_add(int(counts)));
    if (threadIdx.x == 0) sh.equal = cta;
    sync_cluster<C>();
    for (uint32_t r = 0; r < rank; ++r) before += *peer(&sh.equal, r);
    sync_cluster<C>();  // the last read of another CTA's memory
  }
  if (before <= p.rank && p.rank - before < mine) {
    uint32_t left = p.rank - before;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const uint32_t hit = __ballot_sync(0xffffffffu, i0 + lane < w1 && key_of_f32(row.x[min(i0 + lane, w1 - 1)]) == p.key);
      const uint32_t here = __popc(hit);
      if (left < here) {
        if (((hit >> lane) & 1u) && uint32_t(__popc(hit & ((1u << lane) - 1))) == left) {
          g.token[m] = begin + i0 + lane;
          if (g.prob) g.prob[m] = share_of(f32_of_key(p.key), row.top, row.slope, sh.exp2, kept);
        }
        break;
      }
      left -= here;
    }
  }
  pdl_launch_dependents();
}

template <int C>
cudaError_t launch_rows(const Args& g, cudaStream_t s) {
  const int smem = int(sizeof(Shared)) + (g.copy ? g.chunk * 4 : 0);
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t e = raise_smem_cap(sample_f32_kernel<C>, dev, int(kMaxShared));  // one limit for every chunk
  if (e != cudaSuccess) return e;
  return launch_clusters<C>(sample_f32_kernel<C>, g.M * C, kThreads, smem, s, g);
}

}  // namespace

cudaError_t launch_sample_f32(const SampleArgs& args, cudaStream_t s) {
  auto fits = [&](int c) { return sizeof(Shared) + size_t((args.V + c - 1) / c) * 4 <= kMaxShared; };
  // Measured with top-k and top-p: 20 us beside the passes in one CTA, 26 in a cluster; 0.65 ns per logit of a
  // chunk in shared memory, 1 ns from L2.
  int c = ctas_per_row(args.M, [&](int c) {
    return (c == 1 ? 20000.0 : 26000.0) + (fits(c) ? 0.65 : 1.0) * double(args.V) / c;
  });
  while ((args.V + c - 1) / c > kMaxChunk) c *= 2;
  SampleArgs g = args;
  g.chunk = int((g.V + c - 1) / c);
  g.copy = fits(c);
  if (g.M * c > 0x7fffffff) return cudaErrorInvalidConfiguration;
  switch (c) {
    case 1: return launch_rows<1>(g, s);
    case 2: return launch_rows<2>(g, s);
    case 4: return launch_rows<4>(g, s);
    default: return launch_rows<8>(g, s);
  }
}

}  // namespace bl
