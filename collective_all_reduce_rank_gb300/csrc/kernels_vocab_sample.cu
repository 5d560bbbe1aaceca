// kernels_vocab_sample.cu -- tokens drawn from vocabulary-parallel logits.
//
//   w_j = exp((l_j - max l) / temperature); top-k keeps the k largest logits,
//   top-p of those the shortest run of falling logits whose weight reaches p
//   times theirs, min-p what weighs at least min_p (equal logits: the lowest
//   index first); the token is the first index i with
//   sum_{j <= i, kept} w_j > uniform * sum_{kept} w_j
//
// No sort: the bounds of top-k and top-p are found as the logit at which a
// count or a weight is reached, by counting elements in up to 1024 bins over the
// logits' bits as ordered integers: of the nearest 16 octaves of weight first
// (only if the bound is not there, of the others: most logits are far down and
// are then not counted), then of ever narrower ranges, until a bin is one value;
// equal logits at the bound are taken by index.
//
// Weights are integers in units of 2^-44 of the largest, exact sums of which
// depend on no order, so that rows give the same token however many CTAs share
// them.  A weight is within 2^-29 of its value, relative, or a unit; below
// 2^-44 it is zero, and such tokens are never drawn.
//
// A cluster of up to 8 CTAs shares a row.  Each keeps its slice of the logits
// in shared memory, so HBM is read once; histograms and sums are read across
// the cluster.
//
// One row of 131072 bf16 takes 12 to 14 us without bounds, 14 to 25 with them
// and 6 if it is greedy: up to some ten meetings of the cluster, one after
// another.  256 such rows take 134 us, of which 10 are HBM: 68 instructions an
// element, issued in 43% of the cycles, and the meetings.  33 rows of 50021
// float32 take 42: a search of float32 keys narrows two or three times where
// bfloat16's ends after one.  (Two CTAs an SM leave 64 registers a thread, of
// which a few words are spilled: 96 bytes stored, 140 to 160 loaded.)
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
constexpr int kBatch = 4;  // units of a thread whose loads are in flight together
constexpr int kMaxSplit = 8;
constexpr int kUnitBits = 44;
constexpr float kNear = 16.f;  // octaves of weight searched first
constexpr float kFar = 44.f;   // logits further down weigh nothing
constexpr size_t kMostSlice = 184 * 1024;
static_assert((kSampleMaxVocab / kMaxSplit + 1) * 4 + kMaxRanks * 64 <= kMostSlice, "a row fits a cluster");

// 2^(-i / 64) in units of 2^-44; all but the first in [1/2, 1), and that one as
// the largest number below 1, so that its leading bits are a float's.
constexpr int kPowers = 64;
struct PowerTable {
  unsigned long long p[kPowers];
};

constexpr PowerTable make_table() {  // by the series of the exponential
  PowerTable t{};
  for (int i = 0; i < kPowers; ++i) {
    const double x = -(double)i / kPowers * 0.693147180559945309417232121458;
    double sum = 1.0, term = 1.0;
    for (int k = 1; k < 30; ++k) {
      term = term * x / k;
      sum += term;
    }
    t.p[i] = i ? (unsigned long long)(sum * (double)(1ull << kUnitBits) + 0.5) : (1ull << kUnitBits) - 1;
  }
  return t;
}

__device__ const PowerTable kTable = make_table();
constexpr int kCopies = 16;  // of the table: lanes l and l + 16 read the l-th, free of bank conflicts

struct Seg {
  int pos;          // position of its first logit in the slice
  int end;          // one past its last
  long long index;  // vocabulary index of its first logit
};

struct Shared {
  unsigned long long power[kPowers * kCopies];
  Seg seg[kMaxRanks];
  // by parity of the row, read by the cluster
  uint32_t top[2];              // the slice's largest key, all ones if it holds a NaN
  int first[2];                 // position of the first logit equal to the row's maximum
  unsigned long long above[2];  // weight of what is kept in the end, without the bound's ties
  uint32_t ties[2];
  unsigned long long all[2];    // by parity of the histogram: a weight summed beside it
  // of this CTA
  unsigned long long warp_above[2][kWarps];
  uint32_t warp_ties[2][kWarps];
  uint32_t wmax[kWarps];
  unsigned long long scan[kWarps];
  int cut;
  uint32_t allow;
  unsigned long long before, after;
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
  static __device__ __forceinline__ uint32_t from(float f) { return key(__float_as_uint(f)); }  // smallest key >= f
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
  static __device__ __forceinline__ uint32_t from(float f) {
    const uint32_t b = __float_as_uint(f);
    return key(b & 0x80000000u ? b >> 16 : (b + 0xFFFFu) >> 16);
  }
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

// The positions of a unit whose logits lie in a range of keys, as bits: bit(j)
// for the j-th, pos() back.  NaN, a position without a logit, is in none.  A
// range that ends with the key of -0, which no logit has, ends below it: as a
// value it would take in 0, whose key is behind the range.
template <int DT>
struct Within;
template <>
struct Within<RRA_FLOAT32> {
  float lo, hi;
  __device__ __forceinline__ Within(uint32_t from, uint32_t to)
      : lo(Logit<RRA_FLOAT32>::value(from)), hi(Logit<RRA_FLOAT32>::value(to - (to == 0x7FFFFFFFu ? 1 : 0))) {}
  static __device__ __forceinline__ int bit(int j) { return j; }
  static __device__ __forceinline__ int pos(int i) { return i; }
  __device__ __forceinline__ uint32_t up(const uint4& x) const {  // from lo on
    return (__uint_as_float(x.x) >= lo ? 1u : 0u) | (__uint_as_float(x.y) >= lo ? 2u : 0u) |
           (__uint_as_float(x.z) >= lo ? 4u : 0u) | (__uint_as_float(x.w) >= lo ? 8u : 0u);
  }
  __device__ __forceinline__ uint32_t both(const uint4& x) const {
    return up(x) & ((__uint_as_float(x.x) <= hi ? 1u : 0u) | (__uint_as_float(x.y) <= hi ? 2u : 0u) |
                    (__uint_as_float(x.z) <= hi ? 4u : 0u) | (__uint_as_float(x.w) <= hi ? 8u : 0u));
  }
};
// bfloat16: two positions a comparison, so even ones from bit 0 on, odd ones
// from bit 16 on (one at a time a unit's mask took 45 instructions, not 16).
template <>
struct Within<RRA_BFLOAT16> {
  __nv_bfloat162 lo, hi;
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t key) {
    return __float2bfloat162_rn(Logit<RRA_BFLOAT16>::value(key));
  }
  __device__ __forceinline__ Within(uint32_t from, uint32_t to) : lo(two(from)), hi(two(to - (to == 0x7FFFu ? 1 : 0))) {}
  static __device__ __forceinline__ int bit(int j) { return j / 2 + 16 * (j & 1); }
  static __device__ __forceinline__ int pos(int i) { return 2 * (i & 15) + (i >> 4); }
  static __device__ __forceinline__ __nv_bfloat162 pair(const uint32_t& w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return (a & 0x10001u) | (b & 0x20002u) | (c & 0x40004u) | (d & 0x80008u);
  }
  __device__ __forceinline__ uint32_t up(const uint4& x) const {
    return bits(__hge2_mask(pair(x.x), lo), __hge2_mask(pair(x.y), lo), __hge2_mask(pair(x.z), lo),
                __hge2_mask(pair(x.w), lo));
  }
  __device__ __forceinline__ uint32_t both(const uint4& x) const {
    return up(x) & bits(__hle2_mask(pair(x.x), hi), __hle2_mask(pair(x.y), hi), __hle2_mask(pair(x.z), hi),
                        __hle2_mask(pair(x.w), hi));
  }
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

// Weights of a row.  x(l) = (top - l) log2(e) / temperature is reduced as the
// difference of two multiples of 1/64 and of what is left of them.
struct Scale {
  float top;     // largest logit
  float hi, lo;  // log2(e) / temperature as a pair
  float low;     // logits below this weigh nothing (x > kFar)
  float near;    // x is up to kNear from here on
  float base;    // subtracted from every logit, exactly
  int k0;        // of the largest: (top - base) log2(e) / temperature = k0 / 64 + g0
  float g0;
};

constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, of up to 22 bits

// v (hi + lo) = k / 64 + g, less g0; k comes as the bits of k + kRound.
__device__ __forceinline__ float reduce(float v, const Scale& c, float g0, int* k) {
  const float u = __fmul_rn(v, c.hi);
  const float ue = __fmaf_rn(v, c.lo, __fmaf_rn(v, c.hi, -u));
  const float t = __fmaf_rn(u, (float)kPowers, kRound);
  *k = __float_as_int(t);
  return __fadd_rn(__fmaf_rn(__fsub_rn(t, kRound), -1.f / kPowers, u), __fsub_rn(ue, g0));
}

__device__ __forceinline__ Scale make_scale(float top, float temperature) {
  Scale c;
  c.top = top;
  c.hi = __fdiv_rn(1.44269502f, temperature);
  c.lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-c.hi, temperature, 1.44269502f), 1.92596303e-8f), temperature);
  if (!(c.hi < 1e38f)) {  // a temperature below 1.5e-38 counts as that
    c.hi = 1e38f;
    c.lo = 0.f;
  }
  // an infinite temperature, or an infinite logit: what weighs anything weighs the same
  if (c.hi == 0.f || top == INFINITY) c.hi = c.lo = 0.f;
  c.low = top == INFINITY ? top : fmaxf(__fsub_rn(top, __fdiv_rn(kFar, c.hi)), -FLT_MAX);
  c.near = top == INFINITY ? top : fmaxf(__fsub_rn(top, __fdiv_rn(kNear, c.hi)), -FLT_MAX);
  // multiples of 1/64 have 22 bits; where the largest logit has more, those that
  // weigh anything are within a factor of two of it
  c.base = fabsf(top) * c.hi > 30000.f && top != INFINITY ? top : 0.f;
  c.g0 = reduce(fminf(top, FLT_MAX) - c.base, c, 0.f, &c.k0);
  return c;
}

// w = 2^-x(l) for l >= low: 2^(-k / 64) from the table and a quartic for the
// rest, cut to units of 2^-44 and put in the middle of the unit cut to.
__device__ __forceinline__ unsigned long long weight(const Shared& sh, const Scale& c, float l) {
  int k;
  const float g = reduce(fminf(l, FLT_MAX) - c.base, c, c.g0, &k);
  k = c.k0 - k;
  const unsigned long long fixed = sh.power[(k & (kPowers - 1)) * kCopies + (threadIdx.x & (kCopies - 1))];
  // (2^g - 1) 2^(-k / 64) in units of 2^-37
  const float real = __uint_as_float(0x51800000u | ((uint32_t)(fixed >> (kUnitBits - 24)) & 0x7FFFFFu));
  const float e = g * fmaf(g, fmaf(g, fmaf(g, 0.00961813f, 0.05550411f), 0.24022651f), 0.69314718f) * real;
  const unsigned long long w = fixed + (long long)__float2int_rn(e) * (1ll << (kUnitBits - 37));
  return (w >> (k / kPowers)) | 1;
}

// Keys lo to hi in bins of 2^shift, the largest first.
struct Range {
  uint32_t lo, hi;
  int shift;
  __device__ __forceinline__ int bins() const { return (int)((hi - lo) >> shift) + 1; }
};

__device__ __forceinline__ Range with_bins(uint32_t lo, uint32_t hi) {
  const uint32_t span = hi - lo;  // (span >> shift) + 1 <= 1024
  return {lo, hi, span < kBins ? 0 : 32 - __clz(span) - 10};
}

// The smallest key of [lo, hi] for which `is` holds (it does from some key on,
// and for hi): 32 probes of the warp at a time.
template <class Is>
__device__ __forceinline__ uint32_t first_key(uint32_t lo, uint32_t hi, Is is) {
  const uint32_t lane = threadIdx.x & 31;
  while (hi > lo) {
    const uint32_t step = (hi - lo) / 32 + 1;  // lo, lo + step, ... up to hi - 1
    const uint64_t at = (uint64_t)lo + (uint64_t)lane * step;
    const uint32_t yes = __ballot_sync(0xffffffffu, at >= hi || is((uint32_t)at));
    const uint32_t n = yes ? __ffs(yes) - 1 : 32;  // probes that say no
    const uint64_t top = (uint64_t)lo + (uint64_t)n * step;
    if (top < hi) hi = (uint32_t)top;
    if (n) lo = lo + (n - 1) * step + 1;
  }
  return lo;
}

// f v for f in [0, 1], exact but for the fraction (up: rounded up).
__device__ __forceinline__ unsigned long long share_of(unsigned long long v, float f, bool up) {
  const uint32_t bits = __float_as_uint(f), ex = bits >> 23;
  const unsigned long long m = ex ? (bits & 0x7FFFFFu) | 0x800000u : bits;
  const int shift = 150 - (int)(ex ? ex : 1);  // f = m 2^-shift, shift >= 23
  const unsigned long long hi = __umul64hi(v, m), lo = v * m;
  unsigned long long q = 0, rest = m && v;
  if (shift < 64) {
    q = (hi << (64 - shift)) | (lo >> shift);
    rest = lo << (64 - shift);
  } else if (shift < 128) {
    q = hi >> (shift - 64);
    rest = lo | (hi & ((1ull << (shift - 64)) - 1));
  }
  return q + (up && rest ? 1 : 0);
}

// The smallest q with q b >= a, for q of up to 20 bits: float32's quotient is
// off by one at most (a 64-bit division is some 100 instructions).
__device__ __forceinline__ unsigned long long divide_up(unsigned long long a, unsigned long long b) {
  unsigned long long q = (unsigned long long)__fdividef((float)a, (float)b);
  while (q * b < a) ++q;
  while (q && (q - 1) * b >= a) --q;
  return q;
}

// What a bound keeps: all keys above `key`, and the first `ties` equal to it.
struct Bound {
  uint32_t key, ties;
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over this lane and the lanes before it.
template <class T>
__device__ __forceinline__ T prefix(T v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// Lanes hold consecutive parts of a row, `sum` of weight and `ties` at the
// bound each, of which `allow` in all are kept at `unit`: the part in which the
// running weight passes `rest`, -1 if none.  Leaves what of rest and allow
// remains for it (as they were if none).
__device__ __forceinline__ int locate(unsigned long long sum, uint32_t ties, unsigned long long unit,
                                      unsigned long long& rest, uint32_t& allow) {
  const uint32_t seen = prefix(ties) - ties, left = allow > seen ? allow - seen : 0;
  const unsigned long long mass = sum + min(ties, left) * unit, upto = prefix(mass);
  const int i = __ffs(__ballot_sync(0xffffffffu, upto > rest)) - 1;
  if (i < 0) return i;
  rest -= __shfl_sync(0xffffffffu, upto - mass, i);
  allow = __shfl_sync(0xffffffffu, left, i);
  return i;
}

template <int DT>
struct Row {
  using L = Logit<DT>;
  using W = Within<DT>;
  static constexpr int PU = Elem<DT>::kPerUnit;
  const uint4* slice;
  int units;
  uint32_t* hist;  // [2][4][kBins]
  Shared& sh;
  Scale c;
  uint32_t most;  // largest key
  int split;
  int flip;
  int& level;  // parity of the histogram in use

  // The smallest key from `low` on that a bound keeps whatever its index.  (What
  // is behind infinity's key is NaN, the end of no range.)
  static __device__ __forceinline__ uint32_t above(const Bound& b, float low) {
    return max(L::from(low), b.key ? b.key + 1 : 0u);
  }

  __device__ __forceinline__ uint32_t* bins() const { return hist + (level & 1) * 4 * kBins; }

  __device__ __forceinline__ uint32_t raw_at(int at) const {
    return PU == 4 ? reinterpret_cast<const uint32_t*>(slice)[at] : reinterpret_cast<const uint16_t*>(slice)[at];
  }

  // f(raw) for every position of a unit.
  template <class F>
  static __device__ __forceinline__ void unit(const uint4& x, F f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < PU; ++j) f(PU == 4 ? w[j] : (w[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
  }

  // f(raw) for the positions of unit u that are in `mask`, few of them: one at a
  // time a lane, so that a warp's steps are those of its fullest lane.
  template <class F>
  __device__ __forceinline__ void picked(int u, uint32_t mask, F f) const {
    while (mask) {
      const int at = u * PU + W::pos(__ffs(mask) - 1);
      mask &= mask - 1;
      f(raw_at(at));
    }
  }

  // The warp's sum of the weights in units [from, to) from key `lo` on, `each`
  // called with every unit: unit by unit, one at a time a lane where they are
  // few, all of a unit's positions side by side where they are many.
  template <class Each>
  __device__ __forceinline__ unsigned long long sum_of(int from, int to, int step, uint32_t lo, Each each) const {
    const W in(lo, lo);
    unsigned long long sum = 0;
    for (int base = from; base < to; base += step) {
      const int u = base + (int)(threadIdx.x & 31);
      uint4 x = make_uint4(~0u, ~0u, ~0u, ~0u);  // no position
      if (u < to) x = slice[u];
      each(x);
      uint32_t mask = in.up(x);
      if (__any_sync(0xffffffffu, __popc(mask) > PU / 2)) {
        int j = 0;
        unit(x, [&](uint32_t raw) {  // without a branch: the weights' steps overlap
          const bool is = mask >> W::bit(j++) & 1;
          const unsigned long long w = weight(sh, c, is ? L::real(raw) : c.top);
          sum += is ? w : 0;
        });
      } else {
        picked(u, mask, [&](uint32_t raw) { sum += weight(sh, c, L::real(raw)); });
        __syncwarp();
      }
    }
    return warp_sum(sum);
  }

  // Clears the bins of a range.
  __device__ __forceinline__ void clear(const Range& r, int words) const {
    uint4* h = reinterpret_cast<uint4*>(bins());
    for (int k = 0; k < words; ++k)
      for (int i = threadIdx.x; i < (r.bins() + 3) / 4; i += kThreads) h[k * (kBins / 4) + i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }

  // The slice's elements in range and above `keep`'s key, counted by bins, or
  // their weights added (words == 3: pieces of 15 bits, whose sums of up to 2^17
  // elements fit a word) and, in a fourth word, they.  many: the range may hold
  // much of the slice, so that counts of full units go side by side (256 x 131072
  // bf16 143 us without, 134 with; in narrow ranges the vote costs 0.5 us).
  __device__ __forceinline__ void fill(const Range& r, const Bound& keep, int words, bool many) const {
    uint32_t* h = bins();
    const W in(max(r.lo, above(keep, c.low)), r.hi);
    const auto count = [&](uint32_t raw) { atomicAdd(h + ((r.hi - L::key(raw)) >> r.shift), 1u); };
    if (words == 1 && many) {
      for (int base = (int)(threadIdx.x & ~31u); base < units; base += kThreads) {
        const int u = base + (int)(threadIdx.x & 31);
        uint4 x = make_uint4(~0u, ~0u, ~0u, ~0u);  // no position
        if (u < units) x = slice[u];
        const uint32_t mask = in.both(x);
        if (__any_sync(0xffffffffu, __popc(mask) > PU / 2)) {
          int j = 0;
          unit(x, [&](uint32_t raw) {
            if (mask >> W::bit(j++) & 1) count(raw);
          });
        } else {
          picked(u, mask, count);
        }
        __syncwarp();
      }
      return;
    }
    for (int u = threadIdx.x; u < units; u += kThreads)
      picked(u, in.both(slice[u]), [&](uint32_t raw) {
        if (words == 1) {
          count(raw);
          return;
        }
        uint32_t* at = h + ((r.hi - L::key(raw)) >> r.shift);
        const unsigned long long w = weight(sh, c, L::real(raw));
        atomicAdd(at, (uint32_t)w & 0x7FFFu);
        if (w >> 15) atomicAdd(at + kBins, (uint32_t)(w >> 15) & 0x7FFFu);
        if (w >> 30) atomicAdd(at + 2 * kBins, (uint32_t)(w >> 30));
        atomicAdd(at + 3 * kBins, 1u);
      });
    __syncwarp();
  }

  // The CTA's sum of the warps' `sum`, published to the cluster with the bins;
  // then the cluster's.
  __device__ __forceinline__ unsigned long long publish(unsigned long long sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) sh.scan[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      sum = warp_sum(lane < kWarps ? sh.scan[lane] : 0);
      if (lane == 0) sh.all[level & 1] = sum;
    }
    cluster_sync();
    return warp_sum(lane < split ? peer_u64(&sh.all[level & 1], lane) : 0);
  }

  // The cluster's sums of this thread's bins 2 tid and 2 tid + 1 of a range.
  __device__ __forceinline__ void gather(const Range& r, int words, unsigned long long* v) const {
    const int n = r.bins(), b = 2 * threadIdx.x;
    v[0] = v[1] = 0;
    if (b >= n) return;
#pragma unroll 1
    for (int k = 0; k < words; ++k) {
      unsigned long long x[kMaxSplit];  // every CTA's words in flight before the first is used
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q) x[q] = q < split ? peer_u64(bins() + k * kBins + b, q) : 0;
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q) {
        v[0] += (x[q] & 0xFFFFFFFFull) << (15 * k);
        v[1] += (x[q] >> 32) << (15 * k);
      }
    }
    if (b + 1 >= n) v[1] = 0;  // not of the range
  }

  // Of a range's bins, two a thread, the one in which the running sum from
  // `above` on reaches `target` (bins() if none); above: the sum before it (all
  // of it); after: the sum with it.  Up to 64 bins are the first warp's alone.
  __device__ __forceinline__ int reach(const Range& r, const unsigned long long* v, unsigned long long& above,
                                       unsigned long long& after, unsigned long long target) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = 2 * threadIdx.x, n = r.bins();
    unsigned long long end = above + prefix(v[0] + v[1]);
    if (n > 64) {
      if (lane == 31) sh.scan[warp] = end - above;
      __syncthreads();
      const unsigned long long upto = prefix(lane < kWarps ? sh.scan[lane] : 0);
      const unsigned long long before = __shfl_sync(0xffffffffu, upto, warp ? warp - 1 : 0);
      if (warp) end += before;
    }
    if (n > 64 || warp == 0) {
      const unsigned long long begin1 = end - v[1], begin0 = begin1 - v[0];
      const bool last = threadIdx.x == (n > 64 ? kThreads : 32) - 1;
      if (begin0 < target && begin1 >= target) {
        sh.cut = b;
        sh.before = begin0;
        sh.after = begin1;
      } else if (begin1 < target && end >= target) {
        sh.cut = b + 1;
        sh.before = begin1;
        sh.after = end;
      } else if (last && end < target) {
        sh.cut = n;
        sh.before = end;
      }
    }
    ++level;
    __syncthreads();
    above = sh.before;
    after = sh.after;
    const int cut = sh.cut;
    __syncthreads();  // they may be set again
    return cut;
  }

  // The bound that keeps all keys from lo on.
  static __device__ __forceinline__ Bound all_from(uint32_t lo) {
    // below zero's key lies that of -0, which no logit has and whose value is not
    // below zero; a range may begin with either
    return {lo == L::key(0u) ? lo - 2 : lo - 1, 0};
  }

  __device__ __forceinline__ Range bin_keys(const Range& r, int b) const {
    const uint32_t hi = r.hi - ((uint32_t)b << r.shift), below = (1u << r.shift) - 1u;
    return with_bins(hi - r.lo > below ? hi - below : r.lo, hi);
  }

  // The keys searched first: the nearest octaves, of bfloat16 as many of them as
  // leave each key a bin of its own.
  __device__ __forceinline__ uint32_t near_key() const {
    const uint32_t k = min(L::from(c.near), most);
    return DT == RRA_BFLOAT16 && most - k >= kBins ? most - (kBins - 1) : k;
  }

  // The bound of the k largest; none if no more than that weigh anything.
  __device__ __forceinline__ Bound largest(unsigned long long k) {
    const uint32_t near = near_key(), low = min(L::from(c.low), most);
    unsigned long long above = 0, after, v[2];
    Range r = with_bins(near, most);
    for (bool wide = low < near, many = true;;) {
      clear(r, 1);
      fill(r, {0, 0}, 1, many);
      cluster_sync();
      gather(r, 1, v);
      const int b = reach(r, v, above, after, k);
      if (b < r.bins()) {
        if (r.shift == 0) return {r.hi - (uint32_t)b, (uint32_t)(k - above)};
        r = bin_keys(r, b);
        if (after == k) return all_from(r.lo);  // the whole bin, often one element
        many = false;
      } else {
        if (!wide) return {0, 0};
        r = with_bins(low, near - 1);
      }
      wide = false;
    }
  }

  // The bound at which the weight of what `keep` leaves reaches a share of its
  // total.  Where a bin is one key, elements are counted and the key's weight
  // multiplied; else their weights are added.
  __device__ __forceinline__ Bound heaviest(const Bound& keep, float share) {
    const uint32_t near = near_key(), low = min(L::from(c.low), most);
    const unsigned long long extra = keep.key ? weight(sh, c, L::value(keep.key)) * keep.ties : 0;
    unsigned long long above = 0, after, target = 0, v[2];
    Range r = with_bins(near, most);
    for (bool first = true, wide = low < near;; first = false) {
      const int words = r.shift ? 3 : 1;
      clear(r, words + (words > 1));
      fill(r, keep, words, first);
      if (first) {
        const unsigned long long all = publish(
            sum_of((threadIdx.x >> 5) * 32, units, kThreads, Row::above(keep, c.low), [](const uint4&) {}));
        const unsigned long long part = share_of(all + extra, share, true);
        target = part ? part : 1;
      } else {
        cluster_sync();
      }
      gather(r, words, v);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = 2 * (int)threadIdx.x + j;
        if (b >= r.bins()) break;
        const Range q = bin_keys(r, b);
        if (r.shift == 0 && v[j]) v[j] *= weight(sh, c, L::value(q.hi));
        if (extra && keep.key >= q.lo && keep.key <= q.hi) v[j] += extra;
      }
      const uint32_t* elements = bins() + 3 * kBins;
      const int b = reach(r, v, above, after, target);
      if (b < r.bins()) {
        if (r.shift == 0) {
          const uint32_t key = r.hi - (uint32_t)b;
          const unsigned long long each = weight(sh, c, L::value(key));
          unsigned long long ties = divide_up(target - above, each);
          if (key == keep.key && ties > keep.ties) ties = keep.ties;
          return {key, (uint32_t)min(ties, 0xFFFFFFFFull)};
        }
        r = bin_keys(r, b);
        const int lane = threadIdx.x & 31;
        uint32_t n = __reduce_add_sync(0xffffffffu, lane < split ? peer_u32(elements + b, lane) : 0);
        if (extra && keep.key >= r.lo && keep.key <= r.hi) n = 2;
        // it is its element that reaches the share; where `keep` ends inside the
        // bin, that is the last one it leaves
        if (n == 1) return keep.key >= r.lo ? keep : all_from(r.lo);
      } else {
        if (!wide) return keep;  // all of it
        r = with_bins(low, near - 1);
      }
      wide = false;
    }
  }

  // Weight and ties of units [from, to), of which this warp's lanes take one
  // after another; every lane gets them.
  __device__ __forceinline__ void weigh(int from, int to, const Bound& keep, float low, unsigned long long& sum,
                                        uint32_t& ties) const {
    const bool tied = keep.key && L::value(keep.key) >= low;
    const W at(keep.key, keep.key);
    ties = 0;
    sum = sum_of(from, to, 32, above(keep, low), [&](const uint4& x) {
      if (tied) ties += __popc(at.both(x));
    });
    ties = __reduce_add_sync(0xffffffffu, ties);
  }

  // The position in units [from, to), of this warp, at which the running weight
  // passes `rest`; w: its weight.
  __device__ __forceinline__ int draw(int from, int to, const Bound& keep, float low, unsigned long long unit_w,
                                      unsigned long long rest, uint32_t allow, unsigned long long& w) const {
    const float bound = keep.key ? L::value(keep.key) : -INFINITY;  // which weighs nothing
    const W in(max(L::from(low), keep.key), keep.key);
    const int lane = threadIdx.x & 31;
    for (int base = from; base < to; base += 32) {
      unsigned long long sum = 0;
      uint32_t ties = 0;
      if (base + lane < to)
        picked(base + lane, in.up(slice[base + lane]), [&](uint32_t raw) {
          const float l = L::real(raw);
          if (l == bound)
            ++ties;
          else
            sum += weight(sh, c, l);
        });
      __syncwarp();
      const int hit = locate(sum, ties, unit_w, rest, allow);
      if (hit >= 0) {  // the unit's positions side by side
        sum = 0;
        ties = 0;
        if (lane < PU) {
          const float l = L::real(raw_at((base + hit) * PU + lane));
          if (l == bound)
            ties = l >= low;
          else if (l > bound && l >= low)
            sum = weight(sh, c, l);
        }
        __syncwarp();
        const int j = locate(sum, ties, unit_w, rest, allow);
        w = __shfl_sync(0xffffffffu, ties ? unit_w : sum, j & 31);
        return (base + hit) * PU + j;
      }
      const uint32_t met = min(__reduce_add_sync(0xffffffffu, ties), allow);
      rest -= warp_sum(sum) + met * unit_w;
      allow -= met;
    }
    return from * PU;  // not reached: the range holds it
  }
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int split) {
  using L = Logit<DT>;
  constexpr int PU = Elem<DT>::kPerUnit, ES = Elem<DT>::kSize;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  uint32_t* hist = reinterpret_cast<uint32_t*>(dyn);
  uint4* slice = reinterpret_cast<uint4*>(dyn + 8 * kBins * 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)split);
  const long long V = a.first[a.n];
  const long long lo = V * rank / split, hi = V * (rank + 1) / split;
  bool fresh = true;
  int level = 0, flip = 0;
  for (size_t row = blockIdx.x / (unsigned)split; row < a.rows; row += gridDim.x / (unsigned)split, flip ^= 1) {
    const float temperature = a.temperature ? a.temperature[row] : 1.f;
    const int k = a.top_k ? a.top_k[row] : 0;
    const float share = a.top_p ? a.top_p[row] : 1.f, least = a.min_p ? a.min_p[row] : 0.f;
    const float uniform = a.uniform[row];
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
      for (int u0 = tid; u0 < n; u0 += kBatch * kThreads) {
        uint4 x[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (u0 + j * kThreads < n) x[j] = ld_stream(src + u0 + j * kThreads);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int u = u0 + j * kThreads;
          if (u >= n) break;
          if (u > 0 && u < n - 1) {
            most.add(x[j]);
            slice[units + u] = x[j];
          } else {
            const int begin = u == 0 ? skip : 0, end = min(skip + len - u * PU, PU);
            most.add(only<DT>(x[j], begin, end, L::kMinusInf));
            slice[units + u] = only<DT>(x[j], begin, end, L::kNone);
          }
        }
      }
      if (tid == 0) sh.seg[nseg] = {units * PU + skip, units * PU + skip + len, from};
      ++nseg;
      units += n;
    }
    if (fresh) {  // behind the first loads
      for (int i = tid; i < kPowers * kCopies; i += kThreads) sh.power[i] = kTable.p[i / kCopies];
      fresh = false;
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, most.top());
    if (lane == 0) sh.wmax[warp] = top;
    if (tid == 0) sh.first[flip] = INT_MAX;
    __syncthreads();
    if (warp == 0) {
      top = __reduce_max_sync(0xffffffffu, sh.wmax[lane % kWarps]);
      if (lane == 0) sh.top[flip] = top;
    }
    cluster_sync();
    top = __reduce_max_sync(0xffffffffu, lane < split ? peer_u32(&sh.top[flip], lane) : 0u);

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
      const float most_l = L::value(top);
      int at = INT_MAX;
      for (int u = tid; u < units && at == INT_MAX; u += kThreads) {
        int j = 0;
        r.unit(slice[u], [&](uint32_t raw) {
          if (L::real(raw) == most_l && at == INT_MAX) at = u * PU + j;
          ++j;
        });
      }
      at = __reduce_min_sync(0xffffffffu, at);
      if (lane == 0 && at != INT_MAX) atomicMin(&sh.first[flip], at);
      cluster_sync();
      const int mine = lane < split ? (int)peer_u32(&sh.first[flip], lane) : INT_MAX;
      const int owner = __ffs(__ballot_sync(0xffffffffu, mine != INT_MAX)) - 1;
      if (rank == owner && tid == 0) {
        at = sh.first[flip];
        int g = 0;
        while (at >= sh.seg[g].end) ++g;
        a.token[row] = sh.seg[g].index + (at - sh.seg[g].pos);
        if (a.logprob) a.logprob[row] = 0.f;
      }
      continue;
    }

    r.c = make_scale(L::value(top), temperature);
    Bound keep{0, 0};
    if (k > 0 && k < V) keep = r.largest((unsigned long long)k);
    if (share < 1.f) keep = r.heaviest(keep, fmaxf(share, 0.f));
    unsigned long long tie_w = keep.key ? weight(sh, r.c, L::value(keep.key)) : 0;
    float low = r.c.low;
    if (least > 0.f) {  // the smallest logit that weighs as much
      const unsigned long long floor_w =
          min(__float2ull_ru(fminf(least, 1.f) * (float)(1ull << kUnitBits)), weight(sh, r.c, r.c.top));
      const uint32_t key = first_key(min(L::from(r.c.low), top), top,
                                     [&](uint32_t q) { return weight(sh, r.c, L::value(q)) >= floor_w; });
      low = fmaxf(low, L::value(key));
      if (tie_w < floor_w) tie_w = 0;
    }

    // weight of each warp's positions, in the order of the vocabulary, of the
    // CTA's, and of the row
    const int per = (units + kThreads - 1) / kThreads * 32;
    int u0 = min(warp * per, units), u1 = min(u0 + per, units);
    unsigned long long sum;
    uint32_t ties;
    r.weigh(u0, u1, keep, low, sum, ties);
    if (lane == 0) {
      sh.warp_above[0][warp] = sum;
      sh.warp_ties[0][warp] = ties;
    }
    __syncthreads();
    if (warp == 0) {
      sum = warp_sum(lane < kWarps ? sh.warp_above[0][lane] : 0);
      ties = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_ties[0][lane] : 0);
      if (lane == 0) {
        sh.above[flip] = sum;
        sh.ties[flip] = ties;
      }
    }
    cluster_sync();
    if (warp == 0) {
      // sum > uniform * total, as integers
      const unsigned long long w = lane < split ? peer_u64(&sh.above[flip], lane) : 0;
      const uint32_t t = lane < split ? peer_u32(&sh.ties[flip], lane) : 0;
      const uint32_t n = __reduce_add_sync(0xffffffffu, t);
      const unsigned long long total = warp_sum(w) + min(n, keep.ties) * tie_w;
      unsigned long long rest = share_of(total, fminf(fmaxf(uniform, 0.f), 1.f), false);
      if (rest >= total) rest = total - 1;
      uint32_t allow = keep.ties;
      const int owner = locate(w, t, tie_w, rest, allow);
      if (lane == 0) {
        sh.cut = owner;
        sh.before = rest;
        sh.allow = allow;
        sh.scan[0] = total;
      }
    }
    __syncthreads();
    if (sh.cut == rank) {  // it falls in this CTA: in which warp's part, and in which sixteenth of that
      unsigned long long rest = sh.before;
      const unsigned long long total = sh.scan[0];
      uint32_t allow = sh.allow;
      const int w0 = locate(lane < kWarps ? sh.warp_above[0][lane] : 0, lane < kWarps ? sh.warp_ties[0][lane] : 0,
                            tie_w, rest, allow);
      u0 = min(w0 * per, units);
      u1 = min(u0 + per, units);
      const int part = (u1 - u0 + kWarps - 1) / kWarps;
      const int v0 = min(u0 + warp * part, u1), v1 = min(v0 + part, u1);
      r.weigh(v0, v1, keep, low, sum, ties);
      if (lane == 0) {
        sh.warp_above[1][warp] = sum;
        sh.warp_ties[1][warp] = ties;
      }
      __syncthreads();
      const int w1 = locate(lane < kWarps ? sh.warp_above[1][lane] : 0, lane < kWarps ? sh.warp_ties[1][lane] : 0,
                            tie_w, rest, allow);
      if (warp == w1) {
        unsigned long long w;
        const int at = r.draw(v0, v1, keep, low, tie_w, rest, allow, w);
        if (lane == 0) {
          int g = 0;
          while (at >= sh.seg[g].end) ++g;
          a.token[row] = sh.seg[g].index + (at - sh.seg[g].pos);
          if (a.logprob) {
            const float t = (float)total;
            a.logprob[row] = 2 * w > total ? log1pf(-(float)(total - w) / t) : logf((float)w / t);
          }
        }
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
  const size_t smem = 8 * kBins * 4 + (slice(split) + 15) / 16 * 16;
  const cudaError_t attr = raise_smem<kern>(8 * kBins * 4 + kMostSlice + 1024);
  if (attr != cudaSuccess) return attr;
  // a cluster a row: rows differ in their work (greedy ones have next to none),
  // and those that end early make room
  size_t clusters = a.rows;
  const size_t most = (size_t)std::max(1, max_ctas_cap() > 0 ? sms / split : INT_MAX / kMaxSplit);
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
