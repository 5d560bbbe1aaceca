// kernels_skinny.cu -- the gated projections and the vocabulary statistics
// of few tokens (at most kSkinnyTokens): a decoding step, or a handful of
// scored tokens.
//
// With T tokens every weight is used T times, so the call is bound by
// reading the weights once: 2 n F D or V D elements.  A tile of the
// tensor-core product (tc_gemm.cuh) holds 16 KB of weights per stage and CTA
// next to as much padding, and 256 weight rows per tile leave some SMs idle;
// here a unit of work is 16 weight rows, so every SM streams to the end.
//
// A CTA's 8 warps split the K axis of its unit (steps of 64 elements, warp w
// every 8th) and add their partial sums through shared memory.  Weights go
// from global memory straight to the registers of mma.sync m16n8k16: the
// sum over k does not care about the order of k, so each lane takes 8
// consecutive elements of a row (one 16-byte load) as the pairs of two
// products, and the tokens (8 per product, read through L1) are taken in the
// same order.  With 4 steps in flight a warp has 8 KB of loads outstanding.
// Measured against the tensor-core tiles: one token through 8 x 1728 gated
// columns of hidden 5120 47 us (6.0 TB/s) against 88, 8 tokens against
// 131072 columns 200 us (6.7 TB/s) against 268.
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

__device__ __forceinline__ void sk_mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 sk_ldg(const void* p, bool stream) {
  uint4 v;
  if (stream)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  else
    v = __ldg(static_cast<const uint4*>(p));
  return v;
}

// Elements [k, k + 8) of a row of `cols`, zeros past its end (or for a null
// row).  VEC: rows start on 16 bytes and cols is a multiple of 8.  Otherwise
// a row starts at any element: the two 16-byte blocks around the 8 elements
// are loaded (the second is the next lane's first) and shifted together;
// near the end of the matrix (`end`), where the second block may lie outside
// it, and at the end of a row the elements are loaded one by one.
template <bool VEC, bool STREAM>
__device__ __forceinline__ uint4 sk_load(const char* row, int k, int cols, const char* end) {
  if (!row || k >= cols) return make_uint4(0u, 0u, 0u, 0u);
  const char* p = row + (size_t)k * 2;
  if constexpr (VEC) {
    return sk_ldg(p, STREAM);
  } else {
    const char* lo = reinterpret_cast<const char*>((uintptr_t)p & ~(uintptr_t)15);
    if (k + 8 > cols || lo + 32 > end) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      for (int i = 0; i < 8 && k + i < cols; ++i)
        w[i >> 1] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << (16 * (i & 1));
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint4 a = sk_ldg(lo, false), b = sk_ldg(lo + 16, false);
    const uint32_t off = (uint32_t)((uintptr_t)p & 15);
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

// The 16 x 8 NT products of one unit: rows r0 (lane / 4) and r1 (8 + lane /
// 4) of this lane, in matrices that end at e0 and e1; each warp leaves its
// share of the K axis in red[warp][16][8 NT].
template <int NT, bool VEC>
__device__ __forceinline__ void sk_unit(const SkinnyArgs& a, const char* r0, const char* e0, const char* r1,
                                        const char* e1, float (*red)[16 * 8 * NT]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int D = a.hidden, steps = (D + kSkStep - 1) / kSkStep;
  const char* xb = static_cast<const char*>(a.x);
  const char* xend = xb + (size_t)a.tokens * D * 2;
  const char* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = n * 8 + g < a.tokens ? xb + (size_t)(n * 8 + g) * D * 2 : nullptr;
  float c[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[n][i] = 0.f;

  for (int s0 = warp; s0 < steps; s0 += kSkWarps * kSkDepth) {
    uint4 w[kSkDepth][4];
#pragma unroll
    for (int u = 0; u < kSkDepth; ++u) {
      const int k = (s0 + u * kSkWarps) * kSkStep + t * 8;
      w[u][0] = sk_load<VEC, true>(r0, k, D, e0);
      w[u][1] = sk_load<VEC, true>(r1, k, D, e1);
      w[u][2] = sk_load<VEC, true>(r0, k + 32, D, e0);
      w[u][3] = sk_load<VEC, true>(r1, k + 32, D, e1);
    }
#pragma unroll
    for (int u = 0; u < kSkDepth; ++u) {
      const int k = (s0 + u * kSkWarps) * kSkStep + t * 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 lo = w[u][2 * h], hi = w[u][2 * h + 1];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 x = sk_load<VEC, false>(xr[n], k + 32 * h, D, xend);
          sk_mma(c[n], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
          sk_mma(c[n], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
        }
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

template <int NT>
__device__ __forceinline__ float sk_total(const float (*red)[16 * 8 * NT], int i) {
  float v = red[0][i];
#pragma unroll
  for (int w = 1; w < kSkWarps; ++w) v += red[w][i];
  return v;
}

// ---------------------------------------------------------------------------
// gated projections
// ---------------------------------------------------------------------------
template <int NT, bool VEC, int ACT>
__global__ void __launch_bounds__(kSkThreads, 2) skinny_gate_kernel(const __grid_constant__ SkinnyArgs a) {
  __shared__ float red[kSkWarps][16 * 8 * NT];
  const int g = (threadIdx.x & 31) >> 2;
  const int per = (a.width + 7) / 8;  // units per rank
  const size_t bytes = (size_t)a.width * a.hidden * 2;
  pdl_wait();
  pdl_next();
  for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
    const int r = u / per, f0 = (u - r * per) * 8;
    const char* gb = static_cast<const char*>(a.w[2 * r]);
    const char* ub = static_cast<const char*>(a.w[2 * r + 1]);
    const size_t at = (size_t)(f0 + g) * a.hidden * 2;
    const bool in = f0 + g < a.width;
    sk_unit<NT, VEC>(a, in ? gb + at : nullptr, gb + bytes, in ? ub + at : nullptr, ub + bytes, red);
    if (threadIdx.x < 8 * 8 * NT) {
      const int token = threadIdx.x / 8, f = threadIdx.x % 8;  // neighbouring threads, neighbouring columns
      const float gv = sk_total<NT>(red, f * 8 * NT + token), uv = sk_total<NT>(red, (8 + f) * 8 * NT + token);
      float unused;
      const float y = gv * gate_sigma<ACT>(gv, &unused) * uv;
      if (token < a.tokens && f0 + f < a.width)
        static_cast<__nv_bfloat16*>(a.out[r])[(size_t)token * a.width + f0 + f] = __float2bfloat16_rn(y);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// vocabulary statistics
// ---------------------------------------------------------------------------
template <int NT, bool VEC>
__global__ void __launch_bounds__(kSkThreads, 2) skinny_lse_kernel(const __grid_constant__ SkinnyArgs a) {
  __shared__ float red[kSkWarps][16 * 8 * NT];
  __shared__ float2 run[16 * 8 * NT];
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const int slot = threadIdx.x / (8 * NT), token = threadIdx.x % (8 * NT);  // row slot of the unit, token
  const bool mine = slot < 16 && token < a.tokens;
  pdl_wait();
  pdl_next();
  long long target = -1;
  if (mine) {
    target = a.targets[token];
    if (target == a.ignore_index) target = -1;
  }
  float m = -INFINITY, s = 0.f;
  for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
    int r = 0;
    while (u >= a.unit0[r + 1]) ++r;
    const long long v0 = (long long)(u - a.unit0[r]) * 16;
    const char* wb = static_cast<const char*>(a.w[r]);
    const long long rows = a.rows[r];
    const char* end = wb + (size_t)rows * a.hidden * 2;
    const char* r0 = v0 + g < rows ? wb + (size_t)(v0 + g) * a.hidden * 2 : nullptr;
    const char* r1 = v0 + g + 8 < rows ? wb + (size_t)(v0 + g + 8) * a.hidden * 2 : nullptr;
    sk_unit<NT, VEC>(a, r0, end, r1, end, red);
    if (mine && v0 + slot < rows) {
      const float l = sk_total<NT>(red, slot * 8 * NT + token);
      if (target == a.col0[r] + v0 + slot) a.hit[token] = l;
      const float nm = fmaxf(m, l);
      if (nm == -INFINITY) {
        if (l != l) s = l;
      } else {
        s = s * expf(m - nm) + expf(l - nm);
        m = nm;
      }
    }
    __syncthreads();
  }
  if (slot < 16) run[threadIdx.x] = make_float2(m, s);
  __syncthreads();
  if (slot == 0 && mine) {
    for (int i = 1; i < 16; ++i) {
      const float2 q = run[i * 8 * NT + token];
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

int skinny_grid(long long units) {
  long long cap = 2ll * device_sms();
  if (max_ctas_cap() > 0 && max_ctas_cap() < cap) cap = max_ctas_cap();
  return (int)(units < cap ? units : cap);
}

template <int NT, bool VEC>
static cudaError_t gate_go(const SkinnyArgs& a, int act, int grid, cudaStream_t s) {
  if (act == RRA_ACT_SILU) return launch_pdl(skinny_gate_kernel<NT, VEC, RRA_ACT_SILU>, grid, kSkThreads, 0, s, a);
  return launch_pdl(skinny_gate_kernel<NT, VEC, RRA_ACT_GELU_TANH>, grid, kSkThreads, 0, s, a);
}

cudaError_t launch_skinny_gate(const SkinnyArgs& a, int act, cudaStream_t s, int* grid) {
  // a CTA per unit: nothing carries over from unit to unit, and the last
  // units spread over all SMs (1728 units on 304 resident CTAs would take 6
  // trips for 5.7)
  *grid = max_ctas_cap() > 0 && max_ctas_cap() < a.units ? max_ctas_cap() : a.units;
  const bool vec = a.hidden % 8 == 0;  // the matrices themselves are 16-byte aligned
  if (a.tokens <= 8) return vec ? gate_go<1, true>(a, act, *grid, s) : gate_go<1, false>(a, act, *grid, s);
  return vec ? gate_go<2, true>(a, act, *grid, s) : gate_go<2, false>(a, act, *grid, s);
}

cudaError_t launch_skinny_lse(const SkinnyArgs& a, cudaStream_t s, int* grid) {
  *grid = skinny_grid(a.units);
  const bool vec = a.hidden % 8 == 0;
  if (a.tokens <= 8)
    return launch_pdl(vec ? skinny_lse_kernel<1, true> : skinny_lse_kernel<1, false>, *grid, kSkThreads, 0, s, a);
  return launch_pdl(vec ? skinny_lse_kernel<2, true> : skinny_lse_kernel<2, false>, *grid, kSkThreads, 0, s, a);
}

}  // namespace rra
