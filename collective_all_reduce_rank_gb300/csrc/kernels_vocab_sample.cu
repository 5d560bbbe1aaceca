// kernels_vocab_sample.cu -- tokens drawn from vocabulary-parallel logits.
//
//   w_j = exp((l_j - max l) / temperature); top-k keeps the k largest logits,
//   top-p of those the shortest run of falling logits whose weight reaches p
//   times theirs, min-p what weighs at least min_p (equal logits: the lowest
//   index first); the token is the first index i with
//   sum_{j <= i, kept} w_j > uniform * sum_{kept} w_j
//
// No sort: the bounds of top-k and top-p are found as the logit at which a
// count or a weight is reached, by histograms of 1024 bins over ever narrower
// ranges (first of the distance to the maximum, then of the logits' bits as
// ordered integers) until a bin is one value; equal logits at the bound are
// then taken by index.
//
// Weights are integers in units of 2^-43 of the largest, exact sums of which
// depend on no order, so that rows give the same token however many CTAs share
// them.  A weight is within 2^-31 of its value, relative (or half a unit): the
// exponent is formed from the logits' exact difference as a pair of float32,
// reduced in 32.32 fixed point, and 2^f comes from a table of 128 and a cubic.
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

struct PowerTable {
  unsigned long long fixed[128];
  float real[128];
};

// 2^((i + 1/2) / 128) by its series, in units of 2^-43 and as float32.
constexpr PowerTable make_table() {
  PowerTable t{};
  for (int i = 0; i < 128; ++i) {
    const double x = (i + 0.5) / 128.0 * 0.693147180559945309417232121458;
    double sum = 1.0, term = 1.0;
    for (int k = 1; k < 30; ++k) {
      term = term * x / k;
      sum += term;
    }
    t.fixed[i] = (unsigned long long)(sum * (double)(1ull << kUnitBits) + 0.5);
    t.real[i] = (float)sum;
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
  unsigned long long fixed[128];
  float real[128];
  Seg seg[kMaxRanks];
  int nseg, npos;
  uint32_t top[2];   // by parity of the row: the slice's largest key, all ones if it holds a NaN
  int first[2];      // position of the first logit equal to the row's maximum
  unsigned long long above[2][kWarps];  // weight kept of each warp's positions, without the bound's ties
  uint32_t ties[2][kWarps];
  unsigned long long all_above[kMaxSplit * kWarps];  // the cluster's
  uint32_t all_ties[kMaxSplit * kWarps];
  uint32_t wmax[kWarps];
  unsigned long long scan[kWarps];
  int cut;
  unsigned long long before, total;
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
  using Raw = uint32_t;
  static constexpr uint32_t kNone = 0xFFFFFFFFu, kMinusInf = 0xFF800000u;
  static __device__ __forceinline__ uint32_t key(uint32_t b) {
    if (b == 0x80000000u) b = 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
  }
  static __device__ __forceinline__ bool nan(uint32_t b) { return (b & 0x7FFFFFFFu) > 0x7F800000u; }
};
template <>
struct Logit<RRA_BFLOAT16> {
  using Raw = uint16_t;
  static constexpr uint32_t kNone = 0xFFFFu, kMinusInf = 0xFF80u;
  static __device__ __forceinline__ uint32_t key(uint32_t b) {
    if (b == 0x8000u) b = 0;
    return b & 0x8000u ? ~b & 0xFFFFu : b | 0x8000u;
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float((k & 0x8000u ? k ^ 0x8000u : ~k & 0xFFFFu) << 16);
  }
  static __device__ __forceinline__ bool nan(uint32_t b) { return (b & 0x7FFFu) > 0x7F80u; }
};

// Weights of a row.
struct Scale {
  float top;     // largest logit
  float hi, lo;  // log2(e) / temperature as a pair
  float bins;    // bins per unit of logit
};

__device__ __forceinline__ unsigned long long weight(const Shared& sh, const Scale& c, float l) {
  if (l == c.top) return 1ull << kUnitBits;
  const float d = __fsub_rn(c.top, l), z = __fsub_rn(d, c.top);
  const float p = __fmul_rn(d, c.hi);
  if (!(p < 44.f)) return 0;
  const float rest = __fadd_rn(__fsub_rn(c.top, __fsub_rn(d, z)), __fsub_rn(-l, z));
  const float pe = __fmaf_rn(rest, c.hi, __fmaf_rn(d, c.lo, __fmaf_rn(d, c.hi, -p)));
  const long long y = -(__float2ll_rn(p * 4294967296.f) + (long long)__float2int_rn(pe * 4294967296.f));
  const uint32_t f = (uint32_t)y;
  const int n = -(int)(y >> 32);
  const uint32_t i = f >> 25;
  const float x = (float)((int)(f & 0x1FFFFFFu) - (1 << 24)) * 1.6138672e-10f;  // log(2) 2^-32
  const float e = x * fmaf(x, fmaf(x, 0.16666667f, 0.5f), 1.f) * sh.real[i];
  const unsigned long long w = sh.fixed[i] + ((long long)__float2int_rn(e * 274877906944.f) << (kUnitBits - 38));
  return n > 0 ? (w + (1ull << (n - 1))) >> n : w;
}

__device__ __forceinline__ int distance_bin(const Scale& c, float l) {
  if (l == c.top) return 0;  // +infinity too
  const float x = __fmul_rn(__fsub_rn(c.top, l), c.bins);
  return x < (float)(kBins - 1) ? (int)x : kBins - 1;
}

// A range of keys searched: its elements' bins, best first.
struct Range {
  uint32_t lo, hi;
  int shift;  // < 0: bins of the distance to the maximum, all keys
};

template <int DT>
__device__ __forceinline__ int bin_of(const Scale& c, const Range& r, uint32_t key) {
  return r.shift < 0 ? distance_bin(c, Logit<DT>::value(key)) : (int)((r.hi - key) >> r.shift);
}

// The keys of distance bin b: distance_bin falls as keys rise.
template <int DT>
__device__ __forceinline__ Range keys_of(const Scale& c, int b, uint32_t most) {
  uint32_t lo = 1, hi = most;  // smallest key whose bin is <= b
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (distance_bin(c, Logit<DT>::value(mid)) <= b)
      hi = mid;
    else
      lo = mid + 1;
  }
  Range r{lo, most, 0};
  uint32_t a = lo, z = most;  // largest key whose bin is >= b
  while (a < z) {
    const uint32_t mid = z - (z - a) / 2;
    if (distance_bin(c, Logit<DT>::value(mid)) >= b)
      a = mid;
    else
      z = mid - 1;
  }
  r.hi = a;
  return r;
}

__device__ __forceinline__ int shift_for(uint32_t lo, uint32_t hi) {
  const uint32_t span = hi - lo;  // bins (span >> shift) + 1 <= 1024
  return span < kBins ? 0 : 32 - __clz(span) - 10;
}

// What a bound keeps: all keys above `key`, and the first `ties` equal to it.
struct Bound {
  uint32_t key;
  unsigned long long ties;
};

template <int DT>
struct Row {
  using L = Logit<DT>;
  const typename L::Raw* slice;
  uint32_t* hist;  // [2][3][kBins]
  Shared& sh;
  Scale c;
  uint32_t most;  // largest key
  int split;
  int& level;  // parity of the histogram in use

  // Add the slice's elements in range to the histogram: ones, or weights.
  __device__ __forceinline__ void count(const Range& r, bool weights, const Bound& keep) {
    uint32_t* h = hist + (level & 1) * 3 * kBins;
    for (int i = threadIdx.x; i < (weights ? 3 : 1) * kBins; i += kThreads) h[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < sh.npos; i += kThreads) {
      const uint32_t key = L::key(slice[i]);
      if (key <= keep.key || key < r.lo || key > r.hi) continue;
      const int b = bin_of<DT>(c, r, key);
      if (weights) {
        const unsigned long long w = weight(sh, c, L::value(key));
        if (w == 0) continue;
        // pieces of 15 bits, whose sums of up to 2^17 elements fit a word
        atomicAdd(h + b, (uint32_t)w & 0x7FFFu);
        if (w >> 15) atomicAdd(h + kBins + b, (uint32_t)(w >> 15) & 0x7FFFu);
        if (w >> 30) atomicAdd(h + 2 * kBins + b, (uint32_t)(w >> 30));
      } else {
        atomicAdd(h + b, 1u);
      }
    }
    cluster_sync();
  }

  // The bin in which the cluster's sum passes `target` (share >= 0: that share
  // of the total, which `target` then becomes); -1 if it does not.
  __device__ __forceinline__ int find(const Range& r, bool weights, const Bound& keep, unsigned long long extra,
                                      unsigned long long& above, unsigned long long& target, double share) {
    const uint32_t* h = hist + (level & 1) * 3 * kBins;
    unsigned long long v[2] = {0, 0};
    const int b0 = 2 * threadIdx.x;
    for (int q = 0; q < split; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[j] += peer_u32(h + b0 + j, q);
        if (weights)
          v[j] += ((unsigned long long)peer_u32(h + kBins + b0 + j, q) << 15) +
                  ((unsigned long long)peer_u32(h + 2 * kBins + b0 + j, q) << 30);
      }
    if (extra && keep.key >= r.lo && keep.key <= r.hi) {
      const int b = bin_of<DT>(c, r, keep.key);
      if (b == b0) v[0] += extra;
      if (b == b0 + 1) v[1] += extra;
    }
    ++level;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned long long sum = prefix(v[0] + v[1]);
    if (lane == 31) sh.scan[warp] = sum;
    if (threadIdx.x == 0) sh.cut = -1;
    __syncthreads();
    unsigned long long base = above;
    for (int w = 0; w < warp; ++w) base += sh.scan[w];
    if (share >= 0.0) {
      unsigned long long total = 0;
      for (int w = 0; w < kWarps; ++w) total += sh.scan[w];
      const double t = ceil(share * (double)total);
      target = t < 1.0 ? 1ull : (unsigned long long)t;
    }
    const unsigned long long end = base + sum;
    const unsigned long long begin0 = end - v[0] - v[1], begin1 = end - v[1];
    if (begin0 < target && begin1 >= target) {
      sh.cut = b0;
      sh.before = begin0;
    } else if (begin1 < target && end >= target) {
      sh.cut = b0 + 1;
      sh.before = begin1;
    }
    __syncthreads();
    const int cut = sh.cut;
    if (cut >= 0) above = sh.before;
    return cut;
  }

  // The bound at which counts (target) or weights (share) are reached among
  // what `keep` leaves; {0, 0}: nowhere, all of it stays.
  __device__ __forceinline__ Bound search(bool weights, const Bound& keep, unsigned long long target, double share) {
    Range r{1, most, -1};
    unsigned long long above = 0;
    const unsigned long long unit = weights && keep.key ? weight(sh, c, L::value(keep.key)) : 0;
    const unsigned long long extra = unit * keep.ties;
    for (;;) {
      count(r, weights, keep);
      const int b = find(r, weights, keep, extra, above, target, share);
      share = -1.0;
      if (b < 0 || (r.shift < 0 && b >= kZeroBin)) return keep;
      if (r.shift == 0) {
        const uint32_t key = r.hi - (uint32_t)b;
        unsigned long long ties = target - above;
        if (weights) {
          const unsigned long long w = weight(sh, c, L::value(key));
          ties = (ties + w - 1) / w;
        }
        if (key == keep.key && ties > keep.ties) ties = keep.ties;
        return {key, ties};
      }
      if (r.shift < 0) {
        r = keys_of<DT>(c, b, most);
      } else {
        const uint32_t hi = r.hi - ((uint32_t)b << r.shift);
        const uint32_t below = (1u << r.shift) - 1u;
        r.lo = hi - r.lo > below ? hi - below : r.lo;
        r.hi = hi;
      }
      r.shift = shift_for(r.lo, r.hi);
    }
  }
};

template <int DT>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleArgs a, int split) {
  using L = Logit<DT>;
  using Raw = typename L::Raw;
  constexpr int PU = Elem<DT>::kPerUnit, ES = Elem<DT>::kSize;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  uint32_t* hist = reinterpret_cast<uint32_t*>(dyn);
  Raw* slice = reinterpret_cast<Raw*>(dyn + 6 * kBins * 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)split);
  const long long V = a.first[a.n];
  const long long lo = V * rank / split, hi = V * (rank + 1) / split;
  if (tid < 128) {
    sh.fixed[tid] = kTable.fixed[tid];
    sh.real[tid] = kTable.real[tid];
  }
  int level = 0, flip = 0;
  for (size_t row = blockIdx.x / (unsigned)split; row < a.rows; row += gridDim.x / (unsigned)split, flip ^= 1) {
    // the slice as it lies in memory, unit by unit, shard after shard
    __syncthreads();
    uint32_t top = 0;
    int pos = 0, nseg = 0;
    for (int q = 0; q < a.n; ++q) {
      const long long from = max(lo, a.first[q]), to = min(hi, a.first[q + 1]);
      if (from >= to) continue;
      const long long vocab = a.first[q + 1] - a.first[q];
      const char* p = static_cast<const char*>(a.logits[q]) + ((long long)row * vocab + from - a.first[q]) * ES;
      const int skip = (int)((uintptr_t)p & 15) / ES, len = (int)(to - from);
      const int units = (skip + len + PU - 1) / PU;
      const uint4* src = reinterpret_cast<const uint4*>(p - skip * ES);
      for (int u = tid; u < units; u += kThreads) {
        const uint4 x = ld_stream(src + u);
        Raw e[PU];
        *reinterpret_cast<uint4*>(e) = x;
#pragma unroll
        for (int j = 0; j < PU; ++j) {
          const int at = u * PU + j - skip;
          if (at < 0 || at >= len) {
            e[j] = (Raw)L::kNone;
          } else {
            top = max(top, L::nan(e[j]) ? 0xFFFFFFFFu : L::key(e[j]));
          }
        }
        *reinterpret_cast<uint4*>(slice + pos + u * PU) = *reinterpret_cast<const uint4*>(e);
      }
      if (tid == 0) sh.seg[nseg] = {pos + skip, pos + skip + len, from};
      ++nseg;
      pos += units * PU;
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) sh.wmax[warp] = top;
    if (tid == 0) {
      sh.nseg = nseg;
      sh.npos = pos;
      sh.first[flip] = INT_MAX;
    }
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, sh.wmax[lane % kWarps]);
    if (tid == 0) sh.top[flip] = top;
    cluster_sync();
    for (int q = 0; q < split; ++q) top = max(top, peer_u32(&sh.top[flip], q));

    const float temperature = a.temperature ? a.temperature[row] : 1.f;
    const int k = a.top_k ? a.top_k[row] : 0;
    if (top == 0xFFFFFFFFu || top <= L::key(L::kMinusInf) || !(temperature >= 0.f)) {
      // a NaN, or nothing but -infinity
      if (rank == 0 && tid == 0) {
        const bool bad = top == 0xFFFFFFFFu || !(temperature >= 0.f);
        a.token[row] = -1;
        if (a.logprob) a.logprob[row] = __uint_as_float(bad ? 0x7FC00000u : 0xFF800000u);
      }
      cluster_sync();
      continue;
    }
    if (temperature == 0.f || k == 1) {
      int at = INT_MAX;
      for (int i = tid; i < pos; i += kThreads)
        if (L::key(slice[i]) == top) {
          at = i;
          break;
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

    Row<DT> r{slice, hist, sh, {}, top, split, level};
    r.c.top = L::value(top);
    const double scale = fmin(1.4426950408889634 / (double)temperature, 1e30);
    r.c.hi = (float)scale;
    r.c.lo = (float)(scale - (double)r.c.hi);
    r.c.bins = r.c.hi * kBinsPerOctave;
    Bound keep{0, 0};
    if (k > 0 && k < V) keep = r.search(false, keep, (unsigned long long)k, -1.0);
    const float share = a.top_p ? a.top_p[row] : 1.f;
    if (share < 1.f) keep = r.search(true, keep, 0, (double)fmaxf(share, 0.f));
    const float least = a.min_p ? a.min_p[row] : 0.f;
    const double lw = ceil(fmin((double)fmaxf(least, 0.f), 1.0) * (double)(1ull << kUnitBits));
    const unsigned long long floor_w = (unsigned long long)lw;
    unsigned long long tie_w = keep.key ? weight(sh, r.c, L::value(keep.key)) : 0;
    if (tie_w < floor_w) tie_w = 0;

    // weight of each warp's positions, in the order of the vocabulary
    const int per = (pos + kThreads - 1) / kThreads * 32;
    const int p0 = min(warp * per, pos), p1 = min(p0 + per, pos);
    unsigned long long sum = 0;
    uint32_t ties = 0;
    for (int i = p0 + lane; i < p1; i += 32) {
      const uint32_t key = L::key(slice[i]);
      if (key > keep.key && key) {
        const unsigned long long w = weight(sh, r.c, L::value(key));
        if (w >= floor_w) sum += w;
      } else if (key == keep.key && key) {
        ++ties;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
      sh.above[flip][warp] = sum;
      sh.ties[flip][warp] = ties;
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
    const double u = fmin(fmax((double)a.uniform[row], 0.0), 1.0);
    unsigned long long target = (unsigned long long)(u * (double)total);  // sum > u total, as integers
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
      for (int i0 = p0; i0 < p1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < p1 ? L::key(slice[i]) : 0;
        const bool tie = key && key == keep.key;
        const uint32_t before = __popc(__ballot_sync(0xffffffffu, tie) & ((1u << lane) - 1u));
        unsigned long long w = 0;
        if (tie) {
          w = before < allow ? tie_w : 0;
        } else if (key > keep.key) {
          w = weight(sh, r.c, L::value(key));
          if (w < floor_w) w = 0;
        }
        const unsigned long long upto = prefix(w);
        const uint32_t hit = __ballot_sync(0xffffffffu, run + upto > rest);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            int g = 0;
            while (i >= sh.seg[g].end) ++g;
            a.token[row] = sh.seg[g].index + (i - sh.seg[g].pos);
            if (a.logprob) {
              const float t = (float)total;
              a.logprob[row] = 2 * w > total ? log1pf(-(float)(total - w) / t) : logf((float)w / t);
            }
          }
          break;
        }
        run += __shfl_sync(0xffffffffu, upto, 31);
        const uint32_t met = __popc(__ballot_sync(0xffffffffu, tie));
        allow = allow > met ? allow - met : 0;
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
