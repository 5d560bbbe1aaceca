// kernels_skinny.cu -- the gated projections and the vocabulary statistics
// of few tokens (at most 16): a decoding step, or a handful of scored tokens.
//
// With T tokens every weight is used T times, so the call is bound by
// reading the weights once: 2 n F D or V D elements.  A tile of the
// tensor-core product (tc_gemm.cuh) holds 16 KB of weights per stage and CTA
// next to as much padding, and 256 weight rows per tile leave some SMs idle;
// here a unit of work is 16 weight rows, so every SM streams to the end.
//
// KW of a CTA's 8 warps split the K axis of a unit (steps of 64 elements,
// warp w every KW-th) and add their partial sums through shared memory; the
// CTA has 8 / KW units at a time, so that short rows keep loads in flight too
// (split_k).  Weights go from global memory straight to the registers of
// mma.sync m16n8k16: the sum over k does not care about the order of k, so
// each lane takes 8 consecutive elements of a row (one 16-byte load) as the
// pairs of two products, and the tokens (8 per product, read through L1) are
// taken in the same order.  With 4 steps in flight a warp has 8 KB of loads
// outstanding.
// Measured against the tensor-core tiles, us: one token through 8 x 1728
// gated columns of hidden 5120 / 1024 / 128 45 / 6.8 / 3.3 against 55 / 14 /
// 7.9 (6.3 TB/s at 5120); 8 tokens against 131072 columns 200 / 49 / 14
// against 204 / 51 / 24 (6.7 TB/s), against 5000 columns 17 / 9 / 8 against
// 30 / 13 / 9.
//
// Gated: rows 0-7 of a unit are gate rows, rows 8-15 the same 8 up rows, so
// a lane's accumulators hold g and u of one element.  Loss: 16 vocabulary
// rows; each thread keeps the running maximum and sum of its row slot over
// all units of the CTA, and one part per CTA and token is written.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act.cuh"
#include "pdl.cuh"
#include "tc_host.h"

namespace rra {

constexpr int kSkWarps = 8;
constexpr int kSkThreads = 32 * kSkWarps;
constexpr int kSkStep = 64;  // K elements per warp step
constexpr int kSkDepth = 4;  // steps in flight per warp

// Two products, of the first and the last two words of each lane's 16 bytes.
// All lanes take part at once: the loads before branch by lane.
__device__ __forceinline__ void sk_mma2(float* c, uint4 lo, uint4 hi, uint4 x) {
  __syncwarp();
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%10,%11,%12,%13}, {%14,%15}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(lo.x), "r"(hi.x), "r"(lo.y), "r"(hi.y), "r"(x.x), "r"(x.y), "r"(lo.z), "r"(hi.z), "r"(lo.w), "r"(hi.w),
        "r"(x.z), "r"(x.w));
}

// Rows that are not whole 16-byte units (VEC false) start on any element,
// but rows v, v + 8, v + 16, ... of a matrix start at the same offset from 16
// bytes.  A unit then takes such rows, and its K axis is counted from the
// 16-byte block in which they start: position k of the unit is element k -
// off, off = (v cols) mod 8.  Weights are loaded as aligned blocks all the
// same; only the tokens, which all rows share, are shifted.  (With rows side
// by side, each of them shifted from two blocks, 8 tokens against 131072
// columns of hidden 1027 took 154 us.)

// Weight positions [k, k + 8) of a row at `row` (its first element), zeros
// outside the row (or for a null row).  The blocks that hold a row's first
// and last elements hold bytes of the matrix, so no load leaves it but inside
// such a block.
template <bool VEC>
__device__ __forceinline__ uint4 sk_weights(const char* row, int k, int off, int cols) {
  const int e = k - off;
  if (!row || e >= cols) return make_uint4(0u, 0u, 0u, 0u);
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(row + (long long)e * 2));
  if (!VEC && (e < 0 || e + 8 > cols)) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j < 0 || e + j >= cols) w[j >> 1] &= j & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

// Token elements [k, k + 8) of a row that starts anywhere, zeros outside it.
// The two 16-byte blocks around the 8 elements are loaded (both hold elements
// of the row) and shifted together.
template <bool VEC>
__device__ __forceinline__ uint4 sk_tokens(const char* row, int k, int cols) {
  if (!row || k >= cols) return make_uint4(0u, 0u, 0u, 0u);
  const char* p = row + (long long)k * 2;
  if constexpr (VEC) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    if (k < 0 || k + 8 > cols) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i >= 0 && k + i < cols)
          w[i >> 1] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << (16 * (i & 1));
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint32_t off = (uint32_t)((uintptr_t)p & 15);
    const uint4* lo = reinterpret_cast<const uint4*>(p - off);
    const uint4 a = __ldg(lo);
    if (off == 0) return a;
    const uint4 b = __ldg(lo + 1);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t sh = (off & 2) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                      __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
  }
}

// The 16 x 8 NT products of the unit of this warp's group of KW: rows r0
// (lane / 4) and r1 (8 + lane / 4) of this lane, at offset `off`; each warp
// leaves its share of the K axis in red[warp][16][8 NT].
template <int NT, bool VEC, int KW>
__device__ __forceinline__ void sk_unit(const SkinnyArgs& a, const char* r0, const char* r1, int off,
                                        float (*red)[16 * 8 * NT]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int D = a.hidden;
  if (VEC) off = 0;
  const int steps = (D + off + kSkStep - 1) / kSkStep;
  const char* xb = static_cast<const char*>(a.x);
  const char* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = n * 8 + g < a.tokens ? xb + (size_t)(n * 8 + g) * D * 2 : nullptr;
  float c[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[n][i] = 0.f;

  for (int s0 = warp % KW; s0 < steps; s0 += KW * kSkDepth) {
    uint4 w[kSkDepth][4];
#pragma unroll
    for (int u = 0; u < kSkDepth; ++u) {
      const int k = (s0 + u * KW) * kSkStep + t * 8;
      w[u][0] = sk_weights<VEC>(r0, k, off, D);
      w[u][1] = sk_weights<VEC>(r1, k, off, D);
      w[u][2] = sk_weights<VEC>(r0, k + 32, off, D);
      w[u][3] = sk_weights<VEC>(r1, k + 32, off, D);
    }
#pragma unroll
    for (int u = 0; u < kSkDepth; ++u) {
      const int k = (s0 + u * KW) * kSkStep + t * 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          sk_mma2(c[n], w[u][2 * h], w[u][2 * h + 1], sk_tokens<VEC>(xr[n], k + 32 * h - off, D));
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* o = red[warp] + g * 8 * NT + n * 8 + 2 * t;
    o[0] = c[n][0];
    o[1] = c[n][1];
    o[8 * 8 * NT] = c[n][2];
    o[8 * 8 * NT + 1] = c[n][3];
  }
  __syncthreads();
}

// Value i of the unit of group `slot`.
template <int NT, int KW>
__device__ __forceinline__ float sk_total(const float (*red)[16 * 8 * NT], int slot, int i) {
  float v = red[slot * KW][i];
#pragma unroll
  for (int w = 1; w < KW; ++w) v += red[slot * KW + w][i];
  return v;
}

// ---------------------------------------------------------------------------
// gated projections
// ---------------------------------------------------------------------------
// Row i (of 8) of unit u: 8 rows side by side, or every 8th of 64.
template <bool VEC>
__device__ __forceinline__ int sk_gate_row(int u, int i) {
  return VEC ? u * 8 + i : u / 8 * 64 + u % 8 + 8 * i;
}

template <int NT, bool VEC, int KW, int ACT>
__global__ void __launch_bounds__(kSkThreads, 2) skinny_gate_kernel(const __grid_constant__ SkinnyArgs a) {
  constexpr int SLOTS = kSkWarps / KW, PER = 8 * 8 * NT;  // units at a time, values per unit
  __shared__ float red[kSkWarps][16 * 8 * NT];
  const int g = (threadIdx.x & 31) >> 2, mine = (threadIdx.x >> 5) / KW;
  const int per = sk_gate_units(a.width, VEC);
  pdl_wait();
  for (int u0 = blockIdx.x * SLOTS; u0 < a.units; u0 += gridDim.x * SLOTS) {
    {
      const int u = u0 + mine, r = u / per, f = sk_gate_row<VEC>(u - r * per, g);
      const bool in = u < a.units && f < a.width;
      const char* gb = static_cast<const char*>(in ? a.w[2 * r] : nullptr);
      const char* ub = static_cast<const char*>(in ? a.w[2 * r + 1] : nullptr);
      const size_t at = (size_t)f * a.hidden * 2;
      sk_unit<NT, VEC, KW>(a, in ? gb + at : nullptr, in ? ub + at : nullptr,
                           (int)((uint32_t)sk_gate_row<VEC>(u - r * per, 0) * (uint32_t)a.hidden & 7u), red);
    }
#pragma unroll
    for (int i0 = 0; i0 < SLOTS * PER; i0 += kSkThreads) {
      const int i = i0 + threadIdx.x;
      if (SLOTS * PER % kSkThreads != 0 && i >= SLOTS * PER) break;
      const int slot = i / PER, token = i % PER / 8, f = i % 8;  // neighbouring threads, neighbouring columns
      const int u = u0 + slot, r = u / per, col = sk_gate_row<VEC>(u - r * per, f);
      if (u >= a.units || token >= a.tokens || col >= a.width) continue;
      const float gv = sk_total<NT, KW>(red, slot, f * 8 * NT + token);
      const float uv = sk_total<NT, KW>(red, slot, (8 + f) * 8 * NT + token);
      float unused;
      static_cast<__nv_bfloat16*>(a.out[r])[(size_t)token * a.width + col] =
          __float2bfloat16_rn(gv * gate_sigma<ACT>(gv, &unused) * uv);
    }
    __syncthreads();
  }
  pdl_next();
}

// ---------------------------------------------------------------------------
// vocabulary statistics
// ---------------------------------------------------------------------------
// Row i (of 16) of unit u of a shard: side by side, or every 8th of 128.
template <bool VEC>
__device__ __forceinline__ long long sk_loss_row(int u, int i) {
  return VEC ? (long long)u * 16 + i : (long long)(u / 8) * 128 + u % 8 + 8 * i;
}

template <int NT, bool VEC, int KW>
__global__ void __launch_bounds__(kSkThreads, 2) skinny_lse_kernel(const __grid_constant__ SkinnyArgs a) {
  constexpr int SLOTS = kSkWarps / KW, PER = 16 * 8 * NT;             // units at a time, values per unit
  constexpr int EACH = (SLOTS * PER + kSkThreads - 1) / kSkThreads;  // values per thread
  __shared__ float red[kSkWarps][PER];
  __shared__ float2 run[kSkThreads];
  const int lane = threadIdx.x & 31, g = lane >> 2, mine = (threadIdx.x >> 5) / KW;
  // value i of the CTA's units: slot i / PER, row i % PER / (8 NT), token i % (8 NT); a thread's
  // values are kSkThreads apart and so of one token
  const int token = threadIdx.x % (8 * NT);
  long long target = -1;
  pdl_wait();
  if (token < a.tokens) {
    target = a.targets[token];
    if (target == a.ignore_index) target = -1;
  }
  float m = -INFINITY, s = 0.f;
  for (int u0 = blockIdx.x * SLOTS; u0 < a.units; u0 += gridDim.x * SLOTS) {
    {
      const int u = u0 + mine;
      int r = 0;
      while (r + 1 < kMaxRanks && u >= a.unit0[r + 1]) ++r;
      const long long v0 = sk_loss_row<VEC>(u - a.unit0[r], g), v1 = sk_loss_row<VEC>(u - a.unit0[r], g + 8);
      const long long rows = u < a.units ? a.rows[r] : 0;
      const char* wb = static_cast<const char*>(a.w[r]);
      sk_unit<NT, VEC, KW>(a, v0 < rows ? wb + (size_t)v0 * a.hidden * 2 : nullptr,
                           v1 < rows ? wb + (size_t)v1 * a.hidden * 2 : nullptr,
                           (int)((uint32_t)sk_loss_row<VEC>(u - a.unit0[r], 0) * (uint32_t)a.hidden & 7u), red);
    }
    float l[EACH];
    float q = -INFINITY;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int i = j * kSkThreads + threadIdx.x, slot = i / PER, u = u0 + slot;
      l[j] = -INFINITY;
      if (i < SLOTS * PER && u < a.units && token < a.tokens) {
        int r = 0;
        while (u >= a.unit0[r + 1]) ++r;
        const long long v = sk_loss_row<VEC>(u - a.unit0[r], i % PER / (8 * NT));
        if (v < a.rows[r]) {
          l[j] = sk_total<NT, KW>(red, slot, i % PER);
          if (target == a.col0[r] + v) a.hit[token] = l[j];
        }
      }
      q = fmaxf(q, l[j]);
    }
    const float nm = fmaxf(m, q);
    if (nm == -INFINITY) {
#pragma unroll
      for (int j = 0; j < EACH; ++j)
        if (l[j] != l[j]) s = l[j];
    } else {
      s *= expf(m - nm);
#pragma unroll
      for (int j = 0; j < EACH; ++j) s += expf(l[j] - nm);
      m = nm;
    }
    __syncthreads();
  }
  pdl_next();
  run[threadIdx.x] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x < 8 * NT && token < a.tokens) {
    for (int i = token + 8 * NT; i < kSkThreads; i += 8 * NT) {
      const float2 q = run[i];
      const float nm = fmaxf(m, q.x);
      if (nm == -INFINITY) {
        s += q.y;
      } else {
        s = s * expf(m - nm) + q.y * expf(q.x - nm);
        m = nm;
      }
    }
    a.part[(long long)blockIdx.x * a.tokens + token] = make_float2(m, s);
  }
}

// ---------------------------------------------------------------------------

int skinny_most(long long units) {
  const long long cap = 2ll * device_sms();
  return (int)(units < cap ? units : cap);
}

int skinny_grid(long long units) { return budget((size_t)skinny_most(units)); }

// Warps that share a row: the smallest power of two that leaves each at most
// 2 kSkDepth steps of it and, where there are few units, fills the SMs.
// (Measured, 8 tokens: 131072 columns of hidden 128 / 512 with 1 and 1 warps
// 14 and 31 us, with 8 27 and 45; 5000 columns of hidden 512 with 1 warp 10
// us, with 8 8.)
static int split_k(int hidden, int units) {
  const int steps = (hidden + kSkStep - 1) / kSkStep;
  int kw = 1;
  while (kw < kSkWarps && (kw * 2 * kSkDepth < steps ||
                           (kw < steps && (long long)units * kw < 2ll * device_sms() * kSkWarps)))
    kw *= 2;
  return kw;
}

template <int NT, bool VEC, int KW>
static cudaError_t gate_kw(const SkinnyArgs& a, int act, int* grid, cudaStream_t s) {
  // a CTA per group of units: nothing carries over from one to the next, and
  // the last ones spread over all SMs (1728 units on 304 resident CTAs would
  // take 6 trips for 5.7)
  const int groups = (a.units + kSkWarps / KW - 1) / (kSkWarps / KW);
  *grid = max_ctas_cap() > 0 && max_ctas_cap() < groups ? max_ctas_cap() : groups;
  if (act == RRA_ACT_SILU)
    return launch_pdl(skinny_gate_kernel<NT, VEC, KW, RRA_ACT_SILU>, *grid, kSkThreads, 0, s, a);
  return launch_pdl(skinny_gate_kernel<NT, VEC, KW, RRA_ACT_GELU_TANH>, *grid, kSkThreads, 0, s, a);
}

template <int NT, bool VEC, int KW>
static cudaError_t lse_kw(const SkinnyArgs& a, int act, int* grid, cudaStream_t s) {
  (void)act;
  return launch_pdl(skinny_lse_kernel<NT, VEC, KW>, *grid, kSkThreads, 0, s, a);
}

#define SK_PICK(fn, NT, VEC)                                  \
  switch (split_k(a.hidden, a.units)) {                       \
    case 1: return fn<NT, VEC, 1>(a, act, grid, s);           \
    case 2: return fn<NT, VEC, 2>(a, act, grid, s);           \
    case 4: return fn<NT, VEC, 4>(a, act, grid, s);           \
    default: return fn<NT, VEC, 8>(a, act, grid, s);          \
  }

#define SK_LAUNCH(fn)                                                                   \
  const bool vec = a.hidden % 8 == 0; /* the matrices themselves are 16-byte aligned */ \
  if (a.tokens <= 8) {                                                                  \
    if (vec) {                                                                          \
      SK_PICK(fn, 1, true)                                                              \
    } else {                                                                            \
      SK_PICK(fn, 1, false)                                                             \
    }                                                                                   \
  } else if (vec) {                                                                     \
    SK_PICK(fn, 2, true)                                                                \
  } else {                                                                              \
    SK_PICK(fn, 2, false)                                                               \
  }

cudaError_t launch_skinny_gate(const SkinnyArgs& a, int act, cudaStream_t s, int* grid) { SK_LAUNCH(gate_kw) }

cudaError_t launch_skinny_lse(const SkinnyArgs& a, cudaStream_t s, int* grid) {
  const int act = 0;
  *grid = skinny_grid(a.units);
  SK_LAUNCH(lse_kw)
}

#undef SK_PICK
#undef SK_LAUNCH

}  // namespace rra
