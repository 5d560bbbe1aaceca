// kernels_norm8.cu -- the fused all-reduce + RMSNorm with an 8-bit
// checkpoint of the sum, and its backward pass from the checkpoint.
//
//   s = sum_k x_k (float32, ascending ranks), q = 1 / sqrt(mean s^2 + eps),
//   y = s q gamma
//   checkpoint, per block of 128 columns: b = bfloat16(s), e the smallest
//   integer with max |b| <= 448 2^e, code = e4m3(b 2^-e), scale byte e + 127
//   backward: dy = sum_k dy_k, h = (code 2^e) q, w = dy gamma,
//   ds = q (w - h mean(w h)),  dgamma = sum over rows of dy h
//
// e4m3 keeps 4 significant bits over a block's whole range (a block whose
// largest column is 1000 times the others keeps the others), and a
// power-of-two scale makes x 2^-e exact, so rounding to e4m3 is the only
// loss.  s is rounded to bfloat16 first: every border between two codes is a
// bfloat16 value, so a last-bit difference of the float32 sum cannot move a
// code (only a rounding border of bfloat16 itself could).
//
// All three kernels are bound by HBM: each input byte is read once, each
// output byte written once; the float32 row stays in shared memory between
// the two passes over a row.
#include <cuda_fp8.h>

#include "common.cuh"
#include "tc_host.h"

namespace rra {

constexpr int kN8Threads = 256;

struct Save8Args {
  const void* in[kMaxRanks];
  void* out[kMaxRanks];
  const void* gamma;
  uint8_t* codes;
  uint8_t* scales;
  float* rstd;
  size_t rows, hidden;
  float eps;
};

struct Back8Args {
  const void* in[kMaxRanks];
  void* out[kMaxRanks];
  const void* gamma;
  const uint8_t* codes;
  const uint8_t* scales;
  const float* rstd;
  float* part;  // [CTA][hidden] float32: this CTA's rows' share of dgamma
  size_t rows, hidden;
};

template <int DT>
__device__ __forceinline__ void unit_floats(uint4 v, float* f) {
  Acc a;
  acc_init<DT>(a, v);
#pragma unroll
  for (int i = 0; i < Elem<DT>::kPerUnit; ++i) f[i] = __uint_as_float(a.w[i]);
}

// Block reduction in a fixed order; every thread gets the sum.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kN8Threads / 32; ++w) t += part[w];
  return t;
}

// Smallest e in [-127, 120] with amax <= 448 * 2^e (448 = 1.75 * 2^8), amax
// finite and not negative.
__device__ __forceinline__ int ckpt_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - ((b & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return e < -127 ? -127 : e;
}

__device__ __forceinline__ float pow2(int e) {  // e in [-127, 127]
  return e == -127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

// The two codes of two float32 values of at most 448 (NaN where not finite).
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 values2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Codes of one unit (8 or 4 columns) from column u * PU of a row.
template <int DT>
__device__ __forceinline__ void load_codes(const uint8_t* row, size_t u, int valid, bool vec, float* f) {
  constexpr int PU = Elem<DT>::kPerUnit;
  const uint8_t* p = row + u * PU;
  uint32_t w[2] = {0u, 0u};
  if (vec && valid == PU) {
    if constexpr (PU == 8) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = q.x;
      w[1] = q.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  } else {
    for (int i = 0; i < valid; ++i) w[i >> 2] |= (uint32_t)__ldg(p + i) << (8 * (i & 3));
  }
#pragma unroll
  for (int i = 0; i < PU; i += 2) {
    const float2 v = values2((w[i >> 2] >> (8 * (i & 3))) & 0xFFFFu);
    f[i] = v.x;
    f[i + 1] = v.y;
  }
}

template <int N, int DT, bool VEC>
__global__ void __launch_bounds__(kN8Threads) norm_save8_kernel(const __grid_constant__ Save8Args a) {
  constexpr int PU = Elem<DT>::kPerUnit;
  constexpr int ES = Elem<DT>::kSize;
  constexpr int LANES = kCkptBlock / PU;  // lanes that hold one block
  extern __shared__ float srow[];
  __shared__ float s_part[kN8Threads / 32];
  const size_t hidden = a.hidden;
  const size_t units = (hidden + PU - 1) / PU;
  const size_t row = blockIdx.x;
  const size_t row_off = row * hidden * ES;
  const size_t nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  const int tid = threadIdx.x;
  uint8_t* crow = a.codes + row * hidden;
  const bool cvec = VEC && hidden % PU == 0;

  float ss = 0.f;
  for (size_t u0 = 0; u0 < units; u0 += kN8Threads) {
    const size_t u = u0 + tid;
    const int v = u < units ? unit_valid<DT>(u, hidden) : 0;
    float f[PU];
    if (v) {
      uint4 x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = load_in<DT, VEC>(static_cast<const char*>(a.in[k]) + row_off, u, v);
      Acc s;
      acc_init<DT>(s, x[0]);
#pragma unroll
      for (int k = 1; k < N; ++k) acc_add<DT>(s, x[k]);
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        f[i] = i < v ? __uint_as_float(s.w[i]) : 0.f;
        srow[u * PU + i] = f[i];
        ss = __fmaf_rn(f[i], f[i], ss);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PU; ++i) f[i] = 0.f;
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < PU; ++i) {
      f[i] = __bfloat162float(__float2bfloat16_rn(f[i]));
      const float m = fabsf(f[i]);
      if (m <= 3.3895314e38f) top = fmaxf(top, m);  // finite
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (v) {
      const int e = ckpt_exponent(top);
      const float mul = pow2(-e);
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < PU; i += 2) {
        const float lo = fabsf(f[i]) <= 3.3895314e38f ? f[i] * mul : NAN;
        const float hi = fabsf(f[i + 1]) <= 3.3895314e38f ? f[i + 1] * mul : NAN;
        w[i >> 2] |= codes2(lo, hi) << (8 * (i & 3));
      }
      uint8_t* c = crow + u * PU;
      if (cvec && v == PU) {
        if constexpr (PU == 8)
          *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(c) = w[0];
      } else {
        for (int i = 0; i < v; ++i) c[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
      }
      if (u % LANES == 0) a.scales[row * nblk + u / LANES] = (uint8_t)(e + 127);
    }
  }
  const float tot = block_sum(ss, s_part);
  const float inv = rsqrtf(tot / (float)hidden + a.eps);
  if (tid == 0) a.rstd[row] = inv;

  for (size_t u = tid; u < units; u += kN8Threads) {
    const int v = unit_valid<DT>(u, hidden);
    float g[PU];
    unit_floats<DT>(load_in<DT, VEC>(a.gamma, u, v), g);
    Acc y;
#pragma unroll
    for (int i = 0; i < PU; ++i) y.w[i] = __float_as_uint(__fmul_rn(__fmul_rn(srow[u * PU + i], inv), g[i]));
    const uint4 o = acc_narrow<DT>(y);
#pragma unroll
    for (int r = 0; r < N; ++r) store_out<DT, VEC, true>(static_cast<char*>(a.out[r]) + row_off, u, v, o);
  }
}

// out = code 2^e, times rstd of the row and gamma of the column where given.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kN8Threads)
    norm_restore8_kernel(const uint8_t* codes, const uint8_t* scales, const float* rstd, const void* gamma, void* out,
                         size_t rows, size_t hidden) {
  constexpr int PU = Elem<DT>::kPerUnit;
  const size_t units = (hidden + PU - 1) / PU;
  const size_t nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  const bool cvec = VEC && hidden % PU == 0;
  for (size_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float q = rstd ? __ldg(rstd + row) : 1.f;
    for (size_t u = threadIdx.x; u < units; u += kN8Threads) {
      const int v = unit_valid<DT>(u, hidden);
      float f[PU], g[PU];
      load_codes<DT>(codes + row * hidden, u, v, cvec, f);
      if (gamma) unit_floats<DT>(load_in<DT, VEC>(gamma, u, v), g);
      const float mul = pow2((int)__ldg(scales + row * nblk + u * PU / kCkptBlock) - 127);
      Acc y;
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        float t = __fmul_rn(__fmul_rn(f[i], mul), q);
        if (gamma) t = __fmul_rn(t, g[i]);
        y.w[i] = __float_as_uint(t);
      }
      store_out<DT, VEC, true>(static_cast<char*>(out) + row * hidden * Elem<DT>::kSize, u, v, acc_narrow<DT>(y));
    }
  }
}

// A CTA takes every gridDim-th row and keeps its rows' share of dgamma in
// its row of `part` (each thread the columns of its own units, so no atomics
// and a fixed order of the sum).
template <int N, int DT, bool VEC>
__global__ void __launch_bounds__(kN8Threads) norm_back8_kernel(const __grid_constant__ Back8Args a) {
  constexpr int PU = Elem<DT>::kPerUnit;
  constexpr int ES = Elem<DT>::kSize;
  extern __shared__ float srow[];  // the summed gradient of the row
  __shared__ float s_part[2][kN8Threads / 32];
  const size_t hidden = a.hidden;
  const size_t units = (hidden + PU - 1) / PU;
  const size_t nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  const bool cvec = VEC && hidden % PU == 0;
  float* dg = a.part + (size_t)blockIdx.x * hidden;
  int flip = 0;
  bool first = true;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1, first = false) {
    const size_t row_off = row * hidden * ES;
    const float q = __ldg(a.rstd + row);
    const uint8_t* crow = a.codes + row * hidden;
    const uint8_t* srow8 = a.scales + row * nblk;
    float acc = 0.f;
    for (size_t u = threadIdx.x; u < units; u += kN8Threads) {
      const int v = unit_valid<DT>(u, hidden);
      uint4 x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = load_in<DT, VEC>(static_cast<const char*>(a.in[k]) + row_off, u, v);
      float f[PU], g[PU];
      load_codes<DT>(crow, u, v, cvec, f);
      unit_floats<DT>(load_in<DT, VEC>(a.gamma, u, v), g);
      const float mul = pow2((int)__ldg(srow8 + u * PU / kCkptBlock) - 127);
      Acc s;
      acc_init<DT>(s, x[0]);
#pragma unroll
      for (int k = 1; k < N; ++k) acc_add<DT>(s, x[k]);
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        if (i >= v) break;
        const float dy = __uint_as_float(s.w[i]);
        const float h = __fmul_rn(__fmul_rn(f[i], mul), q);
        srow[u * PU + i] = dy;
        acc = __fmaf_rn(__fmul_rn(dy, g[i]), h, acc);
        float* d = dg + u * PU + i;
        *d = first ? dy * h : __fmaf_rn(dy, h, *d);
      }
    }
    const float mean = block_sum(acc, s_part[flip]) / (float)hidden;
    for (size_t u = threadIdx.x; u < units; u += kN8Threads) {
      const int v = unit_valid<DT>(u, hidden);
      float f[PU], g[PU];
      load_codes<DT>(crow, u, v, cvec, f);
      unit_floats<DT>(load_in<DT, VEC>(a.gamma, u, v), g);
      const float mul = pow2((int)__ldg(srow8 + u * PU / kCkptBlock) - 127);
      Acc y;
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        const float h = __fmul_rn(__fmul_rn(f[i], mul), q);
        const float w = i < v ? __fmul_rn(srow[u * PU + i], g[i]) : 0.f;
        y.w[i] = __float_as_uint(__fmul_rn(q, __fmaf_rn(-h, mean, w)));
      }
      const uint4 o = acc_narrow<DT>(y);
#pragma unroll
      for (int r = 0; r < N; ++r) store_out<DT, VEC, true>(static_cast<char*>(a.out[r]) + row_off, u, v, o);
    }
  }
}

// dgamma[c] = sum over the CTAs' partial rows, in order: 32 columns x 8
// strided row groups per CTA.
__global__ void __launch_bounds__(256) dgamma_join_kernel(const float* part, int parts, size_t hidden, float* dgamma) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const size_t c = (size_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < hidden)
    for (int i = k; i < parts; i += 8) v += part[(size_t)i * hidden + c];
  red[k][lane] = v;
  __syncthreads();
  if (k == 0 && c < hidden) {
    for (int i = 1; i < 8; ++i) v += red[i][lane];
    dgamma[c] = v;
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

static size_t row_smem(size_t hidden) { return (hidden + 7) / 8 * 8 * sizeof(float); }

template <int N, int DT, bool VEC>
static cudaError_t save_go(const Save8Args& a, cudaStream_t s) {
  static const cudaError_t attr = cudaFuncSetAttribute(norm_save8_kernel<N, DT, VEC>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (attr != cudaSuccess) return attr;
  norm_save8_kernel<N, DT, VEC><<<(unsigned)a.rows, kN8Threads, row_smem(a.hidden), s>>>(a);
  return cudaGetLastError();
}

template <int N, int DT, bool VEC>
static cudaError_t back_go(const Back8Args& a, int ctas, cudaStream_t s) {
  static const cudaError_t attr = cudaFuncSetAttribute(norm_back8_kernel<N, DT, VEC>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (attr != cudaSuccess) return attr;
  norm_back8_kernel<N, DT, VEC><<<ctas, kN8Threads, row_smem(a.hidden), s>>>(a);
  return cudaGetLastError();
}

template <int N>
static cudaError_t save_n(int dt, bool vec, const Save8Args& a, cudaStream_t s) {
  if (dt == RRA_FLOAT32) return vec ? save_go<N, RRA_FLOAT32, true>(a, s) : save_go<N, RRA_FLOAT32, false>(a, s);
  return vec ? save_go<N, RRA_BFLOAT16, true>(a, s) : save_go<N, RRA_BFLOAT16, false>(a, s);
}

template <int N>
static cudaError_t back_n(int dt, bool vec, const Back8Args& a, int ctas, cudaStream_t s) {
  if (dt == RRA_FLOAT32)
    return vec ? back_go<N, RRA_FLOAT32, true>(a, ctas, s) : back_go<N, RRA_FLOAT32, false>(a, ctas, s);
  return vec ? back_go<N, RRA_BFLOAT16, true>(a, ctas, s) : back_go<N, RRA_BFLOAT16, false>(a, ctas, s);
}

cudaError_t launch_norm_save8(int n, int dt, bool vec, const void* const* in, void* const* out, const void* gamma,
                              size_t rows, size_t hidden, float eps, void* codes, void* scales, float* rstd,
                              cudaStream_t s) {
  Save8Args a{};
  for (int r = 0; r < n; ++r) {
    a.in[r] = in[r];
    a.out[r] = out[r];
  }
  a.gamma = gamma;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  a.rstd = rstd;
  a.rows = rows;
  a.hidden = hidden;
  a.eps = eps;
  switch (n) {
    case 1: return save_n<1>(dt, vec, a, s);
    case 2: return save_n<2>(dt, vec, a, s);
    case 3: return save_n<3>(dt, vec, a, s);
    case 4: return save_n<4>(dt, vec, a, s);
    case 5: return save_n<5>(dt, vec, a, s);
    case 6: return save_n<6>(dt, vec, a, s);
    case 7: return save_n<7>(dt, vec, a, s);
    case 8: return save_n<8>(dt, vec, a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_norm_restore8(int dt, bool vec, const void* codes, const void* scales, const float* rstd,
                                 const void* gamma, void* out, size_t rows, size_t hidden, cudaStream_t s) {
  const size_t cap = max_ctas_cap() > 0 ? max_ctas_cap() : (size_t)device_sms() * 8;
  const int grid = (int)(rows < cap ? rows : cap);
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  const uint8_t* e = static_cast<const uint8_t*>(scales);
  if (dt == RRA_FLOAT32) {
    if (vec)
      norm_restore8_kernel<RRA_FLOAT32, true><<<grid, kN8Threads, 0, s>>>(c, e, rstd, gamma, out, rows, hidden);
    else
      norm_restore8_kernel<RRA_FLOAT32, false><<<grid, kN8Threads, 0, s>>>(c, e, rstd, gamma, out, rows, hidden);
  } else {
    if (vec)
      norm_restore8_kernel<RRA_BFLOAT16, true><<<grid, kN8Threads, 0, s>>>(c, e, rstd, gamma, out, rows, hidden);
    else
      norm_restore8_kernel<RRA_BFLOAT16, false><<<grid, kN8Threads, 0, s>>>(c, e, rstd, gamma, out, rows, hidden);
  }
  return cudaGetLastError();
}

int norm_back8_ctas(size_t rows) {
  const size_t cap = 608;  // 4 per SM of 152
  return (int)(rows < cap ? rows : cap);
}

cudaError_t launch_norm_back8(int n, int dt, bool vec, const void* const* grads, void* const* dxs,
                              const void* codes, const void* scales, const float* rstd, const void* gamma,
                              float* dgamma, float* part, size_t rows, size_t hidden, cudaStream_t s) {
  Back8Args a{};
  for (int r = 0; r < n; ++r) {
    a.in[r] = grads[r];
    a.out[r] = dxs[r];
  }
  a.gamma = gamma;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint8_t*>(scales);
  a.rstd = rstd;
  a.part = part;
  a.rows = rows;
  a.hidden = hidden;
  int ctas = norm_back8_ctas(rows);
  if (max_ctas_cap() > 0 && max_ctas_cap() < ctas) ctas = max_ctas_cap();
  cudaError_t e;
  switch (n) {
    case 1: e = back_n<1>(dt, vec, a, ctas, s); break;
    case 2: e = back_n<2>(dt, vec, a, ctas, s); break;
    case 3: e = back_n<3>(dt, vec, a, ctas, s); break;
    case 4: e = back_n<4>(dt, vec, a, ctas, s); break;
    case 5: e = back_n<5>(dt, vec, a, ctas, s); break;
    case 6: e = back_n<6>(dt, vec, a, ctas, s); break;
    case 7: e = back_n<7>(dt, vec, a, ctas, s); break;
    case 8: e = back_n<8>(dt, vec, a, ctas, s); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  dgamma_join_kernel<<<(int)((hidden + 31) / 32), 256, 0, s>>>(part, ctas, hidden, dgamma);
  return cudaGetLastError();
}

}  // namespace rra
