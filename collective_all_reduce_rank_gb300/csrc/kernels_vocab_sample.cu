// kernels_vocab_sample.cu -- tokens drawn from vocabulary-parallel logits.
//
//   w_j = exp((l_j - max l) / temperature); top-k keeps the k largest logits,
//   top-p of those the shortest run of falling logits whose weight reaches p
//   times theirs, min-p what weighs at least min_p (equal logits: the lowest
//   index first); the token is the first index i with
//   sum_{j <= i, kept} w_j > uniform * sum_{kept} w_j
//
// No sort: the bounds of top-k and top-p are found as the logit at which a
// count or a weight is reached, by histograms of 1024 bins: first counts by the
// distance to the maximum, then counts or weights over ever narrower ranges of
// the logits' bits as ordered integers, until a bin is one value; equal logits
// at the bound are taken by index.  The counts by distance also say, to 3%, how
// the weight is spread, so that top-p needs a histogram of weights over a few
// bins only.
//
// Weights are integers in units of 2^-43 of the largest, exact sums of which
// depend on no order, so that rows give the same token however many CTAs share
// them.  A weight is within 2^-31 of its value, relative (or half a unit): the
// exponent is formed from the logits' exact difference as a pair of float32.
// Weights below half a unit (2^-44) are zero, and such tokens are never drawn.
//
// A cluster of up to 8 CTAs shares a row.  Each keeps its slice of the logits
// in shared memory, so HBM is read once; histograms and sums are read across
// the cluster.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "common.cuh"
#include "serve_host.h"
#include "smem_limit.h"

namespace rra {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kMaxSplit = 8;
constexpr int kUnitBits = 43;
constexpr float kBinsPerOctave = 23.f;  // 44 octaves of weight in 1012 bins
constexpr int kZeroBin = 1013;          // weights of bins from here on are zero
constexpr size_t kMostSlice = 184 * 1024;
static_assert((kSampleMaxVocab / kMaxSplit + 1) * 4 + kMaxRanks * 64 <= kMostSlice, "a row fits a cluster");

// 2^(-i / 128), in units of 2^-44 and as float32.
struct Power {
  unsigned long long fixed;
  float real, pad;
};
struct PowerTable {
  Power p[128];
};

constexpr PowerTable make_table() {  // by the series of the exponential
  PowerTable t{};
  for (int i = 0; i < 128; ++i) {
    const double x = -(double)i / 128.0 * 0.693147180559945309417232121458;
    double sum = 1.0, term = 1.0;
    for (int k = 1; k < 30; ++k) {
      term = term * x / k;
      sum += term;
    }
    t.p[i].fixed = (unsigned long long)(sum * (double)(2ull << kUnitBits) + 0.5);
    t.p[i].real = (float)sum;
  }
  return t;
}

__constant__ PowerTable kTable = make_table();

struct Seg {
  int pos;          // position of its first logit in the slice
  int end;          // one past its last
  long long index;  // vocabulary index of its first logit
};

struct Shared {
  Power power[128];
  Seg seg[kMaxRanks];
  // by parity of the row, read by the cluster
  uint32_t top[2];                        // the slice's largest key, all ones if it holds a NaN
  int first[2];                           // position of the first logit equal to the row's maximum
  unsigned long long sums[2][2][kWarps];  // of the search by weight: all that is kept, what lies above its range
  unsigned long long above[2][kWarps];    // weight kept of each warp's positions, without the bound's ties
  uint32_t ties[2][kWarps];
  // of this CTA
  unsigned long long all_above[kMaxSplit * kWarps];
  uint32_t all_ties[kMaxSplit * kWarps];
  uint32_t wmax[kWarps];
  unsigned long long scan[kWarps];
  float low[kWarps], high[kWarps];
  int cut, cut2;
  unsigned long long before;
};

__device__ __forceinline__ uint32_t s32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t peer(uint32_t addr, int cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}

__device__ __forceinline__ uint32_t peer_u32(const void* p, int cta) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer(s32(p), cta)) : "memory");
  return v;
}

__device__ __forceinline__ unsigned long long peer_u64(const void* p, int cta) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(s32(p), cta)) : "memory");
  return v;
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sum over this lane and the lanes before it.
__device__ __forceinline__ unsigned long long prefix(unsigned long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// Logits as integers in the same order (equal zeros alike); 0 is below every
// logit and marks positions without one.
template <int DT>
struct Logit;
template <>
struct Logit<RRA_FLOAT32> {
  static constexpr uint32_t kNone = 0xFFFFFFFFu, kMinusInf = 0xFF800000u;
  static constexpr uint32_t kNan = 0xFFFFFFFFu;  // in the place of a largest key
  static __device__ __forceinline__ uint32_t key(uint32_t b) {
    if (b == 0x80000000u) b = 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
  }
  static __device__ __forceinline__ float real(uint32_t b) { return __uint_as_float(b); }
  // Largest of units, NaN if one is.
  struct Most {
    float m = -INFINITY;
    __device__ __forceinline__ void put(float v) { asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(v)); }
    __device__ __forceinline__ void add(const uint4& x) {
      put(__uint_as_float(x.x));
      put(__uint_as_float(x.y));
      put(__uint_as_float(x.z));
      put(__uint_as_float(x.w));
    }
    __device__ __forceinline__ uint32_t top() const { return m != m ? kNan : key(__float_as_uint(m)); }
  };
};
template <>
struct Logit<RRA_BFLOAT16> {
  static constexpr uint32_t kNone = 0xFFFFu, kMinusInf = 0xFF80u, kNan = 0xFFFFFFFFu;
  static __device__ __forceinline__ uint32_t key(uint32_t b) {
    if (b == 0x8000u) b = 0;
    return b & 0x8000u ? ~b & 0xFFFFu : b | 0x8000u;
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float((k & 0x8000u ? k ^ 0x8000u : ~k & 0xFFFFu) << 16);
  }
  static __device__ __forceinline__ float real(uint32_t b) { return __uint_as_float(b << 16); }
  struct Most {
    uint32_t m = 0xFF80FF80u;
    __device__ __forceinline__ void put(uint32_t v) { asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(v)); }
    __device__ __forceinline__ void add(const uint4& x) {
      put(x.x);
      put(x.y);
      put(x.z);
      put(x.w);
    }
    __device__ __forceinline__ uint32_t top() const {
      const float a = real(m & 0xFFFFu), b = real(m >> 16);
      return a != a || b != b ? kNan : max(key(m & 0xFFFFu), key(m >> 16));
    }
  };
};

// A unit with the positions outside [from, to) set to `raw`.
template <int DT>
__device__ __forceinline__ uint4 only(const uint4& x, int from, int to, uint32_t raw) {
  constexpr int PU = Elem<DT>::kPerUnit, BITS = 128 / PU;
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < PU; ++j)
    if (j < from || j >= to) {
      const int at = j * BITS % 32;
      const uint32_t mask = (BITS == 32 ? ~0u : (1u << (BITS & 31)) - 1u) << at;
      w[j * BITS / 32] = (w[j * BITS / 32] & ~mask) | (raw << at);
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Weights of a row.
struct Scale {
  float top;     // largest logit
  float hi, lo;  // log2(e) / temperature as a pair
  float bins;    // bins per unit of logit
};

// w = 2^-x, x = (top - l) log2(e) / temperature as a pair p + pe: 2^(-k / 128)
// from the table for the k nearest 128 p, and a cubic for the rest.
__device__ __forceinline__ unsigned long long weight(const Shared& sh, const Scale& c, float l) {
  if (l == c.top) return 1ull << kUnitBits;
  const float d = __fsub_rn(c.top, l), z = __fsub_rn(d, c.top);
  const float p = __fmul_rn(d, c.hi);
  if (!(p < 44.f)) return 0;
  const float rest = __fadd_rn(__fsub_rn(c.top, __fsub_rn(d, z)), __fsub_rn(-l, z));  // of the difference
  const float pe = __fmaf_rn(rest, c.hi, __fmaf_rn(d, c.lo, __fmaf_rn(d, c.hi, -p)));
  const float t = __fmaf_rn(p, 128.f, 12582912.f);  // 1.5 * 2^23: rounds to an integer
  const int k = __float_as_int(t) - 0x4B400000;
  const float g = __fadd_rn(__fmaf_rn(__fsub_rn(t, 12582912.f), -1.f / 128.f, p), pe);
  const float y = g * -0.69314718f;
  const uint4 q = *reinterpret_cast<const uint4*>(&sh.power[k & 127]);
  const float e = y * fmaf(y, fmaf(y, 0.16666667f, 0.5f), 1.f) * __uint_as_float(q.z);
  const unsigned long long fixed = ((unsigned long long)q.y << 32) | q.x;
  const unsigned long long w = fixed + ((long long)__float2int_rn(e * 549755813888.f) << (kUnitBits + 1 - 39));
  return ((w >> (k >> 7)) + 1) >> 1;
}

__device__ __forceinline__ int distance_bin(const Scale& c, float l) {
  if (l == c.top) return 0;  // +infinity too
  const float x = __fmul_rn(__fsub_rn(c.top, l), c.bins);
  return x < (float)(kBins - 1) ? (int)x : kBins - 1;
}

// Keys lo to hi in bins of 2^shift, the largest first.
struct Range {
  uint32_t lo, hi;
  int shift;
};

// The smallest key for which `is` holds (it does from some key on, and for
// `hi`), found by the warp 32 probes at a time.
template <class Is>
__device__ __forceinline__ uint32_t first_key(uint32_t lo, uint32_t hi, Is is) {
  const uint32_t lane = threadIdx.x & 31;
  while (hi > lo) {
    const uint32_t step = (hi - lo) / 32 + 1;  // probes lo, lo + step, ... up to hi - 1
    const uint64_t at = (uint64_t)lo + (uint64_t)lane * step;
    const uint32_t yes = __ballot_sync(0xffffffffu, at >= hi || is((uint32_t)at));
    const int n = yes ? __ffs(yes) - 1 : 32;  // probes that say no
    if (n == 0) return lo;
    const uint64_t top = (uint64_t)lo + (uint64_t)n * step;
    lo = lo + (uint32_t)(n - 1) * step + 1;
    if (top < hi) hi = (uint32_t)top;
  }
  return lo;
}

__device__ __forceinline__ Range with_bins(uint32_t lo, uint32_t hi) {
  const uint32_t span = hi - lo;  // (span >> shift) + 1 <= 1024
  return {lo, hi, span < kBins ? 0 : 32 - __clz(span) - 10};
}

// The keys of distance bins a to b (bins fall as keys rise).
template <int DT>
__device__ __forceinline__ Range keys_of(const Scale& c, int a, int b, uint32_t most) {
  const uint32_t lo = first_key(1, most, [&](uint32_t k) { return distance_bin(c, Logit<DT>::value(k)) <= b; });
  if (a == 0) return with_bins(lo, most);
  const uint32_t next = first_key(lo, most, [&](uint32_t k) { return distance_bin(c, Logit<DT>::value(k)) < a; });
  return with_bins(lo, next - 1);
}

// What a bound keeps: all keys above `key`, and the first `ties` equal to it.
struct Bound {
  uint32_t key;
  unsigned long long ties;
};

// Block-wide sum of a pair in warp order; every thread gets it.
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int DT>
struct Row {
  using L = Logit<DT>;
  static constexpr int PU = Elem<DT>::kPerUnit;
  const uint4* slice;
  int units;
  uint32_t* hist;  // [2][3][kBins]
  Shared& sh;
  Scale c;
  uint32_t most;  // largest key
  int split;
  int flip;
  int& level;  // parity of the histogram in use

  __device__ __forceinline__ uint32_t* bins() const { return hist + (level & 1) * 3 * kBins; }

  __device__ __forceinline__ void clear(int words) {
    uint4* h = reinterpret_cast<uint4*>(bins());
    for (int i = threadIdx.x; i < words * kBins / 4; i += kThreads) h[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }

  // f(raw) for every position of the slice, of this thread's units.
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int u = threadIdx.x; u < units; u += kThreads) unit(slice[u], f);
  }

  template <class F>
  static __device__ __forceinline__ void unit(const uint4& x, F f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < PU; ++j) f(PU == 4 ? w[j] : (w[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
  }

  __device__ __forceinline__ void add(uint32_t* h, int b, unsigned long long w) const {
    // pieces of 15 bits, whose sums of up to 2^17 elements fit a word
    atomicAdd(h + b, (uint32_t)w & 0x7FFFu);
    if (w >> 15) atomicAdd(h + kBins + b, (uint32_t)(w >> 15) & 0x7FFFu);
    if (w >> 30) atomicAdd(h + 2 * kBins + b, (uint32_t)(w >> 30));
  }

  // The cluster's sum of this thread's two bins.
  __device__ __forceinline__ void gather(int words, unsigned long long* v) const {
    const uint32_t* h = bins() + 2 * threadIdx.x;
    v[0] = v[1] = 0;
#pragma unroll
    for (int q = 0; q < kMaxSplit; ++q) {
      if (q >= split) break;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (k >= words) break;
        const unsigned long long x = peer_u64(h + k * kBins, q);
        v[0] += (x & 0xFFFFFFFFull) << (15 * k);
        v[1] += (x >> 32) << (15 * k);
      }
    }
  }

  // The bin in which the running sum (from `above` on) reaches `target`, -1 if
  // none; above: the sum before it.
  __device__ __forceinline__ int find(const unsigned long long* v, unsigned long long& above,
                                      unsigned long long target) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned long long sum = prefix(v[0] + v[1]);
    if (lane == 31) sh.scan[warp] = sum;
    if (threadIdx.x == 0) sh.cut = -1;
    __syncthreads();
    unsigned long long end = above + sum;
    for (int w = 0; w < warp; ++w) end += sh.scan[w];
    const unsigned long long begin1 = end - v[1], begin0 = begin1 - v[0];
    if (begin0 < target && begin1 >= target) {
      sh.cut = 2 * threadIdx.x;
      sh.before = begin0;
    } else if (begin1 < target && end >= target) {
      sh.cut = 2 * threadIdx.x + 1;
      sh.before = begin1;
    }
    __syncthreads();
    const int cut = sh.cut;
    if (cut >= 0) above = sh.before;
    __syncthreads();  // sh.cut may be set again
    return cut;
  }

  // Narrows a range of keys to the one key at which the sum reaches `target`:
  // of ones, or of weights (without the elements up to key `at`; `extra` is what
  // is kept of that one's).  The range's bins have been filled and published.
  __device__ __forceinline__ uint32_t narrow(Range r, bool weights, uint32_t at, unsigned long long extra,
                                             unsigned long long& above, unsigned long long target) {
    for (;;) {
      unsigned long long v[2];
      gather(weights ? 3 : 1, v);
      if (extra && at >= r.lo && at <= r.hi) {
        const int b = (int)((r.hi - at) >> r.shift) - 2 * (int)threadIdx.x;
        if (b == 0) v[0] += extra;
        if (b == 1) v[1] += extra;
      }
      ++level;
      const int b = find(v, above, target);
      if (b < 0) return 0;  // not in the range: the callers' targets are
      const uint32_t hi = r.hi - ((uint32_t)b << r.shift);
      if (r.shift == 0) return hi;
      const uint32_t below = (1u << r.shift) - 1u;
      r = with_bins(hi - r.lo > below ? hi - below : r.lo, hi);
      fill(r, weights, at);
    }
  }

  // The slice's elements in range and above key `skip`, counted or weighed.
  __device__ __forceinline__ void fill(const Range& r, bool weights, uint32_t skip) {
    clear(weights ? 3 : 1);
    uint32_t* h = bins();
    each([&](uint32_t raw) {
      const uint32_t key = L::key(raw);
      if (key < r.lo || key > r.hi || key <= skip) return;
      const int b = (int)((r.hi - key) >> r.shift);
      if (weights)
        add(h, b, weight(sh, c, L::value(key)));
      else
        atomicAdd(h + b, 1u);
    });
    cluster_sync();
  }

  // Counts of the bins of distance to the maximum; v: this thread's two.
  __device__ __forceinline__ void count(unsigned long long* v) {
    clear(1);
    uint32_t* h = bins();
    each([&](uint32_t raw) {
      const int b = distance_bin(c, L::real(raw));
      if (b < kZeroBin) atomicAdd(h + b, 1u);  // not a weightless or empty position (NaN)
    });
    cluster_sync();
    gather(1, v);
    ++level;
  }

  // The bound of the k largest; v: counts by distance, cut to them.
  __device__ __forceinline__ Bound largest(unsigned long long* v, unsigned long long k) {
    unsigned long long above = 0;
    const int b = find(v, above, k);
    if (b < 0) return {0, 0};  // no more than k that weigh anything
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 2 * threadIdx.x + j;
      if (i > b) v[j] = 0;
      if (i == b) v[j] = k - above;
    }
    const Range r = keys_of<DT>(c, b, b, most);
    fill(r, false, 0);
    const uint32_t key = narrow(r, false, 0, 0, above, k);
    return {key, k - above};
  }

  // The bound at which the weight of what `keep` leaves reaches a share of its
  // total; v: its counts by distance.  A bin's weights differ by one part in 33,
  // so the counts say in which few bins the bound lies; one pass then sums all
  // weights exactly, those bins' by key.
  __device__ __forceinline__ Bound heaviest(const unsigned long long* v, const Bound& keep, double share) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i0 = 2 * threadIdx.x;
    float hi[2], lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      hi[j] = (float)v[j] * exp2f(-(float)(i0 + j) / kBinsPerOctave);
      lo[j] = (float)v[j] * exp2f(-(float)(i0 + j + 1) / kBinsPerOctave);
    }
    float ph = hi[0] + hi[1], pl = lo[0] + lo[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float a = __shfl_up_sync(0xffffffffu, ph, o), b = __shfl_up_sync(0xffffffffu, pl, o);
      if (lane >= o) {
        ph += a;
        pl += b;
      }
    }
    if (lane == 31) {
      sh.high[warp] = ph;
      sh.low[warp] = pl;
    }
    if (threadIdx.x == 0) {
      sh.cut = kBins - 1;
      sh.cut2 = kBins - 1;
    }
    __syncthreads();
    float th = 0.f, tl = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        ph += sh.high[w];
        pl += sh.low[w];
      }
      th += sh.high[w];
      tl += sh.low[w];
    }
    // 1.001: the sums' own roundings, and the bins' borders
    const float least = (float)share * tl / 1.001f, most_w = (float)share * th * 1.001f;
    if (ph >= least) atomicMin(&sh.cut, ph - hi[1] >= least ? i0 : i0 + 1);
    if (pl >= most_w) atomicMin(&sh.cut2, pl - lo[1] >= most_w ? i0 : i0 + 1);
    __syncthreads();
    const int b1 = max(sh.cut - 1, 0), b2 = min(sh.cut2 + 1, kBins - 1);
    const Range r = keys_of<DT>(c, b1, b2, most);
    clear(3);
    uint32_t* h = bins();
    unsigned long long all = 0, over = 0;
    each([&](uint32_t raw) {
      const uint32_t key = L::key(raw);
      if (key <= keep.key) return;
      const unsigned long long w = weight(sh, c, L::value(key));
      all += w;
      if (key > r.hi)
        over += w;
      else if (key >= r.lo && w)
        add(h, (int)((r.hi - key) >> r.shift), w);
    });
    all = warp_sum(all);
    over = warp_sum(over);
    if (lane == 0) {
      sh.sums[flip][0][warp] = all;
      sh.sums[flip][1][warp] = over;
    }
    cluster_sync();
    const unsigned long long unit = keep.key ? weight(sh, c, L::value(keep.key)) : 0, extra = unit * keep.ties;
    all = over = 0;
    for (int i = lane; i < split * kWarps; i += 32) {
      all += peer_u64(&sh.sums[flip][0][i % kWarps], i / kWarps);
      over += peer_u64(&sh.sums[flip][1][i % kWarps], i / kWarps);
    }
    all = warp_sum(all) + extra;
    over = warp_sum(over) + (keep.key > r.hi ? extra : 0);
    const double t = ceil(share * (double)all);
    const unsigned long long target = t < 1.0 ? 1ull : (unsigned long long)t;
    const uint32_t key = narrow(r, true, keep.key, extra, over, target);
    if (key == 0) return keep;
    const unsigned long long w = weight(sh, c, L::value(key));
    unsigned long long ties = (target - over + w - 1) / w;
    if (key == keep.key && ties > keep.ties) ties = keep.ties;
    return {key, ties};
  }
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int split) {
  using L = Logit<DT>;
  constexpr int PU = Elem<DT>::kPerUnit, ES = Elem<DT>::kSize;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  uint32_t* hist = reinterpret_cast<uint32_t*>(dyn);
  uint4* slice = reinterpret_cast<uint4*>(dyn + 6 * kBins * 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)split);
  const long long V = a.first[a.n];
  const long long lo = V * rank / split, hi = V * (rank + 1) / split;
  if (tid < 128) sh.power[tid] = kTable.p[tid];
  int level = 0, flip = 0;
  for (size_t row = blockIdx.x / (unsigned)split; row < a.rows; row += gridDim.x / (unsigned)split, flip ^= 1) {
    // the slice as it lies in memory, unit by unit, shard after shard
    __syncthreads();
    typename L::Most most;
    int units = 0, nseg = 0;
    for (int q = 0; q < a.n; ++q) {
      const long long from = max(lo, a.first[q]), to = min(hi, a.first[q + 1]);
      if (from >= to) continue;
      const long long vocab = a.first[q + 1] - a.first[q];
      const char* p = static_cast<const char*>(a.logits[q]) + ((long long)row * vocab + from - a.first[q]) * ES;
      const int skip = (int)((uintptr_t)p & 15) / ES, len = (int)(to - from);
      const int n = (skip + len + PU - 1) / PU;
      const uint4* src = reinterpret_cast<const uint4*>(p - skip * ES);
#pragma unroll 4
      for (int u = tid; u < n; u += kThreads) {
        const uint4 x = ld_stream(src + u);
        if (u > 0 && u < n - 1) {
          most.add(x);
          slice[units + u] = x;
        } else {
          const int from = u == 0 ? skip : 0, to = min(skip + len - u * PU, PU);
          most.add(only<DT>(x, from, to, L::kMinusInf));
          slice[units + u] = only<DT>(x, from, to, L::kNone);
        }
      }
      if (tid == 0) sh.seg[nseg] = {units * PU + skip, units * PU + skip + len, from};
      ++nseg;
      units += n;
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, most.top());
    if (lane == 0) sh.wmax[warp] = top;
    if (tid == 0) sh.first[flip] = INT_MAX;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, sh.wmax[lane % kWarps]);
    if (tid == 0) sh.top[flip] = top;
    cluster_sync();
    top = __reduce_max_sync(0xffffffffu, lane < split ? peer_u32(&sh.top[flip], lane) : 0u);

    const float temperature = a.temperature ? a.temperature[row] : 1.f;
    const int k = a.top_k ? a.top_k[row] : 0;
    if (top == L::kNan || top <= L::key(L::kMinusInf) || !(temperature >= 0.f)) {
      // a NaN, or nothing but -infinity
      if (rank == 0 && tid == 0) {
        const bool bad = top == L::kNan || !(temperature >= 0.f);
        a.token[row] = -1;
        if (a.logprob) a.logprob[row] = __uint_as_float(bad ? 0x7FC00000u : 0xFF800000u);
      }
      cluster_sync();
      continue;
    }
    Row<DT> r{slice, units, hist, sh, {}, top, split, flip, level};
    if (temperature == 0.f || k == 1) {
      int at = INT_MAX;
      for (int u = tid; u < units && at == INT_MAX; u += kThreads) {
        int j = 0;
        r.unit(slice[u], [&](uint32_t raw) {
          if (L::key(raw) == top && at == INT_MAX) at = u * PU + j;
          ++j;
        });
      }
      at = __reduce_min_sync(0xffffffffu, at);
      if (lane == 0) atomicMin(&sh.first[flip], at);
      cluster_sync();
      int owner = 0;
      while (owner < split && (int)peer_u32(&sh.first[flip], owner) == INT_MAX) ++owner;
      if (rank == owner && tid == 0) {
        at = sh.first[flip];
        int g = 0;
        while (at >= sh.seg[g].end) ++g;
        a.token[row] = sh.seg[g].index + (at - sh.seg[g].pos);
        if (a.logprob) a.logprob[row] = 0.f;
      }
      continue;
    }

    r.c.top = L::value(top);
    const double scale = fmin(1.4426950408889634 / (double)temperature, 1e30);
    r.c.hi = (float)scale;
    r.c.lo = (float)(scale - (double)r.c.hi);
    r.c.bins = r.c.hi * kBinsPerOctave;
    Bound keep{0, 0};
    const float share = a.top_p ? a.top_p[row] : 1.f;
    if ((k > 0 && k < V) || share < 1.f) {
      unsigned long long v[2];
      r.count(v);
      if (k > 0 && k < V) keep = r.largest(v, (unsigned long long)k);
      if (share < 1.f) keep = r.heaviest(v, keep, (double)fmaxf(share, 0.f));
    }
    const float least = a.min_p ? a.min_p[row] : 0.f;
    const unsigned long long floor_w =
        (unsigned long long)ceil((double)fminf(fmaxf(least, 0.f), 1.f) * (double)(1ull << kUnitBits));
    unsigned long long tie_w = keep.key ? weight(sh, r.c, L::value(keep.key)) : 0;
    if (tie_w < floor_w) tie_w = 0;

    // weight of each warp's positions, in the order of the vocabulary
    const int per = (units + kThreads - 1) / kThreads * 32;
    const int u0 = min(warp * per, units), u1 = min(u0 + per, units);
    const auto kept = [&](uint32_t key) -> unsigned long long {
      if (key <= keep.key) return 0;
      const unsigned long long w = weight(sh, r.c, L::value(key));
      return w < floor_w ? 0 : w;
    };
    unsigned long long sum = 0;
    uint32_t ties = 0;
    for (int u = u0 + lane; u < u1; u += 32)
      r.unit(slice[u], [&](uint32_t raw) {
        const uint32_t key = L::key(raw);
        sum += kept(key);
        ties += key == keep.key;
      });
    sum = warp_sum(sum);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
      sh.above[flip][warp] = sum;
      sh.ties[flip][warp] = keep.key ? ties : 0;
    }
    cluster_sync();
    constexpr int kEach = kMaxSplit * kWarps / 32;  // entries of a lane, in order
    if (tid < kMaxSplit * kWarps) {
      const int q = tid / kWarps, w = tid % kWarps;
      sh.all_above[tid] = q < split ? peer_u64(&sh.above[flip][w], q) : 0;
      sh.all_ties[tid] = q < split ? peer_u32(&sh.ties[flip][w], q) : 0;
    }
    __syncthreads();
    // the ties each warp of the cluster keeps, and where the draw falls
    unsigned long long n = 0, mass[kEach], left[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) n += sh.all_ties[lane * kEach + j];
    unsigned long long seen = prefix(n) - n, mine = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const unsigned long long t = sh.all_ties[lane * kEach + j];
      left[j] = keep.ties > seen ? keep.ties - seen : 0;
      mass[j] = sh.all_above[lane * kEach + j] + min(t, left[j]) * tie_w;
      seen += t;
      mine += mass[j];
    }
    unsigned long long at = prefix(mine);
    const unsigned long long total = __shfl_sync(0xffffffffu, at, 31);
    at -= mine;
    const double u01 = fmin(fmax((double)a.uniform[row], 0.0), 1.0);
    unsigned long long target = (unsigned long long)(u01 * (double)total);  // sum > u total, as integers
    if (target >= total) target = total - 1;
    int owner = -1;
    unsigned long long rest = 0, allow = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (at <= target && at + mass[j] > target) {
        owner = lane * kEach + j;
        rest = target - at;
        allow = left[j];
      }
      at += mass[j];
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, owner >= 0)) - 1;
    owner = __shfl_sync(0xffffffffu, owner, from);
    rest = __shfl_sync(0xffffffffu, rest, from);
    allow = __shfl_sync(0xffffffffu, allow, from);
    if (owner == rank * kWarps + warp) {
      unsigned long long run = 0;
      for (int base = u0; base < u1; base += 32) {
        const int u = base + lane;
        const uint4 x = u < u1 ? slice[u] : make_uint4(~0u, ~0u, ~0u, ~0u);  // no position
        uint32_t met = 0;
        unsigned long long w = 0;
        r.unit(x, [&](uint32_t raw) {
          const uint32_t key = L::key(raw);
          w += kept(key);
          met += keep.key && key == keep.key;
        });
        const unsigned long long before = prefix(met) - met;  // ties of the lanes before
        const unsigned long long mine_left = allow > before ? allow - before : 0;
        w += min((unsigned long long)met, mine_left) * tie_w;
        const unsigned long long upto = prefix(w);
        const uint32_t hit = __ballot_sync(0xffffffffu, run + upto > rest);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            unsigned long long sofar = run + upto - w, ties_left = mine_left;
            int j = 0, found = -1;
            unsigned long long fw = 0;
            r.unit(x, [&](uint32_t raw) {
              const uint32_t key = L::key(raw);
              unsigned long long q = kept(key);
              if (keep.key && key == keep.key && ties_left) {
                --ties_left;
                q = tie_w;
              }
              sofar += q;
              if (found < 0 && sofar > rest) {
                found = u * PU + j;
                fw = q;
              }
              ++j;
            });
            int g = 0;
            while (found >= sh.seg[g].end) ++g;
            a.token[row] = sh.seg[g].index + (found - sh.seg[g].pos);
            if (a.logprob) {
              const float t = (float)total;
              a.logprob[row] = 2 * fw > total ? log1pf(-(float)(total - fw) / t) : logf((float)fw / t);
            }
          }
          break;
        }
        run += __shfl_sync(0xffffffffu, upto, 31);
        const uint32_t all_met = __reduce_add_sync(0xffffffffu, met);
        allow = allow > all_met ? allow - all_met : 0;
      }
    }
  }
  cluster_sync();  // the others may still read this CTA's sums
}

template <int DT>
cudaError_t sample_go(const SampleArgs& a, cudaStream_t s, int* grid_out) {
  constexpr int ES = Elem<DT>::kSize;
  constexpr auto kern = sample_kernel<DT>;
  const size_t V = (size_t)a.first[a.n];
  int sms = device_sms();
  if (max_ctas_cap() > 0 && max_ctas_cap() < sms) sms = max_ctas_cap();
  const auto slice = [&](int split) { return ((V + split - 1) / split + 1) * ES + (size_t)a.n * 64; };
  // the fewest CTAs whose shared memory holds a row; then slices of which two
  // share an SM; then more CTAs a row while there are SMs for them and a slice
  // stays worth its CTA
  int split = 1;
  while (split < kMaxSplit && slice(split) > kMostSlice) split *= 2;
  while (split < kMaxSplit && split * 2 <= sms && slice(split) > 72 * 1024) split *= 2;
  while (split < kMaxSplit && a.rows * split * 2 <= (size_t)sms && V / (split * 2) >= 2048) split *= 2;
  const size_t smem = 6 * kBins * 4 + (slice(split) + 15) / 16 * 16;
  const cudaError_t attr = raise_smem<kern>(6 * kBins * 4 + kMostSlice + 1024);
  if (attr != cudaSuccess) return attr;
  size_t clusters = a.rows;
  const size_t most = (size_t)std::max(1, (max_ctas_cap() > 0 ? sms : 2 * sms) / split);
  if (clusters > most) clusters = most;
  *grid_out = (int)clusters * split;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)*grid_out);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)split;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, split);
}

}  // namespace

cudaError_t launch_vocab_sample(int dt, const SampleArgs& a, cudaStream_t s, int* grid) {
  return dt == RRA_BFLOAT16 ? sample_go<RRA_BFLOAT16>(a, s, grid) : sample_go<RRA_FLOAT32>(a, s, grid);
}

}  // namespace rra
