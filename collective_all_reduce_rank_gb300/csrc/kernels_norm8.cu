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
// output byte written once.  A CTA of 256 threads takes a row; a thread's
// columns are 16-byte units (unit u: thread u mod 256).  Rows of up to 6144
// columns of 16-byte aligned buffers stay in registers between the two
// passes over a row ("reg" kernels, 24 float32 a thread); longer rows, and
// rows that start anywhere, keep the sums in shared memory ("gen" kernels):
// their loads combine the two aligned 16-byte blocks around a unit, their
// stores go through shared memory so that a warp still writes whole words of
// neighbouring columns.
//
// Measured (one GB300, 5120 columns of bfloat16, 8 ranks): forward of 4096
// rows 102 us, 6.2 TB/s of DRAM traffic; backward of 4096 rows 113 us with
// the join of dgamma, 6.1 TB/s of its floor; 1283 x 1027 float32 x 3 ranks
// backward 19 us, 1.8 TB/s (latency: 3 rows a CTA, each a load, a barrier
// and a store).
//
// The sum of squares is added in the order of the kernel that saves nothing
// (kernels_rmsnorm.cu), so that both give the same bits.
#include <cuda_fp8.h>

#include "common.cuh"
#include "pdl.cuh"
#include "smem_limit.h"
#include "tc_host.h"

namespace rra {

constexpr int kN8Threads = 256;
constexpr int kN8MaxThreads = 320;           // backward of long or unaligned rows
constexpr int kN8Regs = 24;                  // float32 of a row a thread keeps
constexpr float kBf16Max = 3.3895314e38f;    // largest finite bfloat16

struct Save8Args {
  const void* in[kMaxRanks];
  void* out[kMaxRanks];
  const void* gamma;
  uint8_t* codes;
  uint8_t* scales;
  float* rstd;
  size_t rows, hidden;
  float eps;
  int vec;
  int stage_codes;
};

struct Back8Args {
  const void* in[kMaxRanks];
  void* out[kMaxRanks];
  const void* gamma;
  const uint8_t* codes;
  const uint8_t* scales;
  const float* rstd;
  float* part;   // [CTA][pitch] float32: this CTA's rows' share of dgamma
  size_t pitch;  // hidden rounded up to whole units
  size_t rows, hidden;
  int vec;
};

template <int DT>
__device__ __forceinline__ void unit_floats(uint4 v, float* f) {
  Acc a;
  acc_init<DT>(a, v);
#pragma unroll
  for (int i = 0; i < Elem<DT>::kPerUnit; ++i) f[i] = __uint_as_float(a.w[i]);
}

// A unit of a row that starts on any element: the aligned 16-byte blocks
// that hold its first and its last byte (both hold bytes of the row), the
// second fetched by the next thread too and so an L1 hit.
template <int DT>
__device__ __forceinline__ uint4 load_any(const char* row, size_t u, int valid) {
  const char* p = row + u * 16;
  if (valid < Elem<DT>::kPerUnit) return ld_partial<DT>(p, valid);
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
  return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh), __funnelshift_r(w[2], w[3], sh),
                    __funnelshift_r(w[3], w[4], sh));
}

template <int DT>
__device__ __forceinline__ uint4 load_row(const char* row, size_t u, int valid, bool vec) {
  return vec ? ld_stream(row + u * 16) : load_any<DT>(row, u, valid);
}

// gamma is read again by every row: kept in L1
template <int DT>
__device__ __forceinline__ void load_gamma(const void* gamma, size_t u, int valid, bool vec, float* f) {
  const char* g = static_cast<const char*>(gamma);
  unit_floats<DT>(vec ? __ldg(reinterpret_cast<const uint4*>(g) + u) : load_any<DT>(g, u, valid), f);
}

// Block reduction in a fixed order; every thread gets the sum.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  if (blockDim.x == kN8Threads) {
#pragma unroll
    for (int w = 0; w < kN8Threads / 32; ++w) t += part[w];
  } else {
    for (int w = 0; w < (int)blockDim.x / 32; ++w) t += part[w];
  }
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

// Codes of one unit (8 or 4 columns), raw.
template <int DT>
__device__ __forceinline__ uint2 load_codes(const uint8_t* row, size_t u, int valid, bool vec) {
  constexpr int PU = Elem<DT>::kPerUnit;
  const uint8_t* p = row + u * PU;
  if (vec) {
    if constexpr (PU == 8) return __ldg(reinterpret_cast<const uint2*>(p));
    return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(p)), 0u);
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < PU; ++i)
    if (i < valid) w[i >> 2] |= (uint32_t)__ldg(p + i) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

template <int DT>
__device__ __forceinline__ void code_floats(uint2 c, float mul, float* f) {
  constexpr int PU = Elem<DT>::kPerUnit;
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < PU; i += 2) {
    const float2 v = values2((w[i >> 2] >> (8 * (i & 3))) & 0xFFFFu);
    f[i] = __fmul_rn(v.x, mul);
    f[i + 1] = __fmul_rn(v.y, mul);
  }
}

// Codes of a unit's sums f, in all lanes of a warp at once: lanes of one
// block of 128 columns share its largest value.  *e gets the block's
// exponent.
template <int DT>
__device__ __forceinline__ uint2 encode_unit(const float* f, int* e) {
  constexpr int PU = Elem<DT>::kPerUnit;
  float b[PU], top = 0.f;
#pragma unroll
  for (int i = 0; i < PU; ++i) {
    b[i] = __bfloat162float(__float2bfloat16_rn(f[i]));
    const float m = fabsf(b[i]);
    top = m <= kBf16Max ? fmaxf(top, m) : top;  // finite
  }
#pragma unroll
  for (int o = kCkptBlock / PU / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  *e = ckpt_exponent(top);
  const float mul = pow2(-*e);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < PU; i += 2) {
    const float lo = fabsf(b[i]) <= kBf16Max ? b[i] * mul : NAN;
    const float hi = fabsf(b[i + 1]) <= kBf16Max ? b[i + 1] * mul : NAN;
    w[i >> 2] |= codes2(lo, hi) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// Ask L2 for the line of unit u of every rank's row that this CTA takes next
// (one lane per 128-byte line): it arrives while the CTA joins and stores the
// present one.
template <int N>
__device__ __forceinline__ void prefetch_ranks(const void* const* in, size_t row_off, size_t u) {
  if ((threadIdx.x & 7) != 0) return;
#pragma unroll
  for (int k = 0; k < N; ++k)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(in[k]) + row_off + u * 16));
}

// The sum over ranks of one unit.
template <int N, int DT>
__device__ __forceinline__ void sum_ranks(const void* const* in, size_t row_off, size_t u, int valid, bool vec, Acc& s) {
  uint4 x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = load_row<DT>(static_cast<const char*>(in[k]) + row_off, u, valid, vec);
  acc_init<DT>(s, x[0]);
#pragma unroll
  for (int k = 1; k < N; ++k) acc_add<DT>(s, x[k]);
}

template <int DT>
__device__ __forceinline__ void put_codes(uint8_t* c, uint2 w, int valid, bool vec) {
  if (vec) {
    if constexpr (Elem<DT>::kPerUnit == 8)
      *reinterpret_cast<uint2*>(c) = w;
    else
      *reinterpret_cast<uint32_t*>(c) = w.x;
  } else {
    const uint32_t q[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < Elem<DT>::kPerUnit; ++i)
      if (i < valid) c[i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
  }
}

// Store a row held in shared memory (unit u's 16 bytes at u * stride) to a
// row of global memory that starts on any element, in 4-byte words.
template <int DT>
__device__ __forceinline__ void store_row_any(char* dst, const char* units, int stride, size_t hidden) {
  if constexpr (Elem<DT>::kSize == 4) {
    for (size_t i = threadIdx.x; i < hidden; i += blockDim.x)
      reinterpret_cast<uint32_t*>(dst)[i] = *reinterpret_cast<const uint32_t*>(units + (i >> 2) * stride + (i & 3) * 4);
  } else {
    auto at = [&](size_t i) { return *reinterpret_cast<const uint16_t*>(units + (i >> 3) * stride + (i & 7) * 2); };
    uint16_t* o = reinterpret_cast<uint16_t*>(dst);
    const size_t head = ((uintptr_t)dst >> 1) & 1;  // one element before the first whole word
    if (threadIdx.x == 0 && head) o[0] = at(0);
    for (size_t i = head + 2 * threadIdx.x; i < hidden; i += 2 * blockDim.x) {
      if (i + 1 < hidden)
        *reinterpret_cast<uint32_t*>(o + i) = (uint32_t)at(i) | ((uint32_t)at(i + 1) << 16);
      else
        o[i] = at(i);
    }
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// A CTA takes a row, or (LOOP: an SM budget leaves fewer CTAs than rows) every
// gridDim-th row.  The loop costs up to 16 registers, so it is a variant.
template <int N, int DT, bool LOOP>
__global__ void __launch_bounds__(kN8Threads) save8_reg_kernel(const __grid_constant__ Save8Args a) {
  constexpr int PU = Elem<DT>::kPerUnit, U = kN8Regs / PU;
  __shared__ float s_part[2][kN8Threads / 32];
  const int units = (int)(a.hidden / PU), tid = threadIdx.x;
  const size_t nblk = (a.hidden + kCkptBlock - 1) / kCkptBlock;
  int flip = 0;
  size_t row = blockIdx.x;
  pdl_wait();
  do {
    const size_t row_off = row * a.hidden * Elem<DT>::kSize;
    float f[U][PU];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (j * kN8Threads >= units) break;
      const int u = j * kN8Threads + tid;
#pragma unroll
      for (int i = 0; i < PU; ++i) f[j][i] = 0.f;
      if (u < units) {
        Acc s;
        sum_ranks<N, DT>(a.in, row_off, u, PU, true, s);
#pragma unroll
        for (int i = 0; i < PU; ++i) {
          f[j][i] = __uint_as_float(s.w[i]);
          ss = __fmaf_rn(f[j][i], f[j][i], ss);
        }
      }
    }
    const float tot = block_sum(ss, s_part[flip]);
    const float inv = rsqrtf(tot / (float)a.hidden + a.eps);
    if (tid == 0) a.rstd[row] = inv;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (j * kN8Threads >= units) break;
      const int u = j * kN8Threads + tid;
      int e;
      const uint2 c = encode_unit<DT>(f[j], &e);
      if (u >= units) continue;
      float g[PU];
      load_gamma<DT>(a.gamma, u, PU, true, g);
      Acc y;
#pragma unroll
      for (int i = 0; i < PU; ++i) y.w[i] = __float_as_uint(__fmul_rn(__fmul_rn(f[j][i], inv), g[i]));
      const uint4 o = acc_narrow<DT>(y);
#pragma unroll
      for (int r = 0; r < N; ++r) st_stream(static_cast<char*>(a.out[r]) + row_off + (size_t)u * 16, o);
      put_codes<DT>(a.codes + row * a.hidden + (size_t)u * PU, c, PU, true);
      if (u % (kCkptBlock / PU) == 0) a.scales[row * nblk + u / (kCkptBlock / PU)] = (uint8_t)(e + 127);
    }
    row += gridDim.x;
    flip ^= 1;
  } while (LOOP && row < a.rows);
  pdl_next();
}

template <int N, int DT, bool LOOP>
__global__ void __launch_bounds__(kN8Threads) save8_gen_kernel(const __grid_constant__ Save8Args a) {
  constexpr int PU = Elem<DT>::kPerUnit;
  extern __shared__ __align__(16) char smem[];  // PU float32 per unit, then (stage_codes) the row's codes
  __shared__ float s_part[2][kN8Threads / 32];
  const size_t hidden = a.hidden, units = (hidden + PU - 1) / PU;
  const size_t nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  const int tid = threadIdx.x;
  uint8_t* cstage = reinterpret_cast<uint8_t*>(smem + units * PU * 4);
  int flip = 0;
  size_t row = blockIdx.x;
  pdl_wait();
  do {
    const size_t row_off = row * hidden * Elem<DT>::kSize;
    uint8_t* crow = a.codes + row * hidden;
    float ss = 0.f;
    for (size_t u0 = 0; u0 < units; u0 += kN8Threads) {
      const size_t u = u0 + tid;
      const int v = u < units ? unit_valid<DT>(u, hidden) : 0;
      float f[PU];
#pragma unroll
      for (int i = 0; i < PU; ++i) f[i] = 0.f;
      if (v) {
        Acc s;
        sum_ranks<N, DT>(a.in, row_off, u, v, a.vec, s);
#pragma unroll
        for (int i = 0; i < PU; ++i) {
          f[i] = i < v ? __uint_as_float(s.w[i]) : 0.f;
          ss = __fmaf_rn(f[i], f[i], ss);
        }
        float4* o = reinterpret_cast<float4*>(smem + u * PU * 4);
#pragma unroll
        for (int i = 0; i < PU / 4; ++i) o[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      }
      int e;
      const uint2 c = encode_unit<DT>(f, &e);
      if (v) {
        if (a.stage_codes)
          put_codes<DT>(cstage + u * PU, c, PU, true);
        else
          put_codes<DT>(crow + u * PU, c, v, a.vec);
        if (u % (kCkptBlock / PU) == 0) a.scales[row * nblk + u / (kCkptBlock / PU)] = (uint8_t)(e + 127);
      }
    }
    const float tot = block_sum(ss, s_part[flip]);
    if (!LOOP || row + gridDim.x >= a.rows) pdl_next();
    const float inv = rsqrtf(tot / (float)hidden + a.eps);
    if (tid == 0) a.rstd[row] = inv;
    for (size_t u = tid; u < units; u += kN8Threads) {
      const int v = unit_valid<DT>(u, hidden);
      float g[PU];
      load_gamma<DT>(a.gamma, u, v, a.vec, g);
      const float* f = reinterpret_cast<const float*>(smem + u * PU * 4);
      Acc y;
#pragma unroll
      for (int i = 0; i < PU; ++i) y.w[i] = __float_as_uint(__fmul_rn(__fmul_rn(f[i], inv), g[i]));
      const uint4 o = acc_narrow<DT>(y);
      if (a.vec) {
#pragma unroll
        for (int r = 0; r < N; ++r) st_stream(static_cast<char*>(a.out[r]) + row_off + u * 16, o);
      } else {
        *reinterpret_cast<uint4*>(smem + u * PU * 4) = o;  // over this thread's own sums
      }
    }
    if (!a.vec) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < N; ++r) store_row_any<DT>(static_cast<char*>(a.out[r]) + row_off, smem, PU * 4, hidden);
      if (a.stage_codes) {  // whole words of the row of bytes
        const size_t head = (4 - ((uintptr_t)crow & 3)) & 3;
        if (tid < head && tid < hidden) crow[tid] = cstage[tid];
        for (size_t i = head + 4 * tid; i < hidden; i += 4 * kN8Threads) {
          if (i + 4 <= hidden)
            *reinterpret_cast<uint32_t*>(crow + i) = (uint32_t)cstage[i] | ((uint32_t)cstage[i + 1] << 8) |
                                                     ((uint32_t)cstage[i + 2] << 16) | ((uint32_t)cstage[i + 3] << 24);
          else
            for (size_t k = i; k < hidden; ++k) crow[k] = cstage[k];
        }
      }
      if (LOOP) __syncthreads();  // the staged row has left
    }
    row += gridDim.x;
    flip ^= 1;
  } while (LOOP && row < a.rows);
}

// out = code 2^e, times rstd of the row and gamma of the column where given.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kN8Threads)
    restore8_kernel(const uint8_t* codes, const uint8_t* scales, const float* rstd, const void* gamma, void* out,
                    size_t rows, size_t hidden) {
  constexpr int PU = Elem<DT>::kPerUnit;
  extern __shared__ __align__(16) char smem[];
  const size_t units = (hidden + PU - 1) / PU;
  const size_t nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  pdl_wait();
  for (size_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float q = rstd ? __ldg(rstd + row) : 1.f;
    char* orow = static_cast<char*>(out) + row * hidden * Elem<DT>::kSize;
    for (size_t u = threadIdx.x; u < units; u += kN8Threads) {
      const int v = VEC ? PU : unit_valid<DT>(u, hidden);
      float f[PU], g[PU];
      code_floats<DT>(load_codes<DT>(codes + row * hidden, u, v, VEC),
                      pow2((int)__ldg(scales + row * nblk + u * PU / kCkptBlock) - 127), f);
      if (gamma) load_gamma<DT>(gamma, u, v, VEC, g);
      Acc y;
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        float t = __fmul_rn(f[i], q);
        if (gamma) t = __fmul_rn(t, g[i]);
        y.w[i] = __float_as_uint(t);
      }
      if constexpr (VEC)
        st_stream(orow + u * 16, acc_narrow<DT>(y));
      else
        *reinterpret_cast<uint4*>(smem + u * 16) = acc_narrow<DT>(y);
    }
    if constexpr (!VEC) {
      __syncthreads();
      store_row_any<DT>(orow, smem, 16, hidden);
      __syncthreads();
    }
  }
  pdl_next();
}

// ---------------------------------------------------------------------------
// backward.  A CTA takes every gridDim-th row; a thread's columns are the
// same in every row, so it adds up its share of dgamma with no atomics and
// in a fixed order, and leaves it in the CTA's row of `part`.
// ---------------------------------------------------------------------------
template <int N, int DT>
__global__ void __launch_bounds__(kN8Threads, 2) back8_reg_kernel(const __grid_constant__ Back8Args a) {
  constexpr int PU = Elem<DT>::kPerUnit, U = kN8Regs / PU;
  __shared__ float s_part[2][kN8Threads / 32];
  const int units = (int)(a.hidden / PU), tid = threadIdx.x;
  const size_t nblk = (a.hidden + kCkptBlock - 1) / kCkptBlock;
  float dg[U][PU];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < PU; ++i) dg[j][i] = 0.f;
  int flip = 0;
  pdl_wait();
  pdl_next();
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const size_t row_off = row * a.hidden * Elem<DT>::kSize;
    const float q = __ldg(a.rstd + row);
    float dy[U][PU], mul[U];
    uint2 code[U];
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (j * kN8Threads >= units) break;
      const int u = j * kN8Threads + tid;
      if (u >= units) continue;
      code[j] = load_codes<DT>(a.codes + row * a.hidden, u, PU, true);
      mul[j] = pow2((int)__ldg(a.scales + row * nblk + u * PU / kCkptBlock) - 127);
      Acc s;
      sum_ranks<N, DT>(a.in, row_off, u, PU, true, s);
      float h[PU], g[PU];
      code_floats<DT>(code[j], mul[j], h);
      load_gamma<DT>(a.gamma, u, PU, true, g);
      if (row + gridDim.x < a.rows)
        prefetch_ranks<N>(a.in, row_off + (size_t)gridDim.x * a.hidden * Elem<DT>::kSize, u);
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        dy[j][i] = __uint_as_float(s.w[i]);
        const float hq = __fmul_rn(h[i], q);
        acc = __fmaf_rn(__fmul_rn(dy[j][i], g[i]), hq, acc);
        dg[j][i] = __fmaf_rn(dy[j][i], hq, dg[j][i]);
      }
    }
    const float mean = block_sum(acc, s_part[flip]) / (float)a.hidden;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (j * kN8Threads >= units) break;
      const int u = j * kN8Threads + tid;
      if (u >= units) continue;
      float h[PU], g[PU];
      code_floats<DT>(code[j], mul[j], h);
      load_gamma<DT>(a.gamma, u, PU, true, g);
      Acc y;
#pragma unroll
      for (int i = 0; i < PU; ++i)
        y.w[i] = __float_as_uint(
            __fmul_rn(q, __fmaf_rn(-__fmul_rn(h[i], q), mean, __fmul_rn(dy[j][i], g[i]))));
      const uint4 o = acc_narrow<DT>(y);
#pragma unroll
      for (int r = 0; r < N; ++r) st_stream(static_cast<char*>(a.out[r]) + row_off + (size_t)u * 16, o);
    }
  }
  float4* part = reinterpret_cast<float4*>(a.part + (size_t)blockIdx.x * a.pitch);
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = j * kN8Threads + tid;
    if (u >= units) continue;
#pragma unroll
    for (int i = 0; i < PU / 4; ++i)
      part[u * (PU / 4) + i] = make_float4(dg[j][4 * i], dg[j][4 * i + 1], dg[j][4 * i + 2], dg[j][4 * i + 3]);
  }
}

template <int N, int DT>
__global__ void __launch_bounds__(kN8MaxThreads, N >= 6 ? 2 : 3) back8_gen_kernel(const __grid_constant__ Back8Args a) {
  constexpr int PU = Elem<DT>::kPerUnit;
  extern __shared__ __align__(16) char smem[];  // PU float32 per unit: the row's summed gradient
  __shared__ float s_part[2][kN8MaxThreads / 32];
  const size_t hidden = a.hidden, units = (hidden + PU - 1) / PU;
  const size_t nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  const int tid = threadIdx.x;
  float4* part = reinterpret_cast<float4*>(a.part + (size_t)blockIdx.x * a.pitch);
  int flip = 0;
  bool first = true;
  pdl_wait();
  pdl_next();
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1, first = false) {
    const size_t row_off = row * hidden * Elem<DT>::kSize;
    const float q = __ldg(a.rstd + row);
    const uint8_t* crow = a.codes + row * hidden;
    const uint8_t* erow = a.scales + row * nblk;
    float acc = 0.f;
    for (size_t u = tid; u < units; u += blockDim.x) {
      const int v = a.vec ? PU : unit_valid<DT>(u, hidden);
      float h[PU], g[PU], d[PU];
      code_floats<DT>(load_codes<DT>(crow, u, v, a.vec), pow2((int)__ldg(erow + u * PU / kCkptBlock) - 127), h);
      load_gamma<DT>(a.gamma, u, v, a.vec, g);
      Acc s;
      sum_ranks<N, DT>(a.in, row_off, u, v, a.vec, s);
      if (row + gridDim.x < a.rows)
        prefetch_ranks<N>(a.in, row_off + (size_t)gridDim.x * hidden * Elem<DT>::kSize, u);
      float4* sm = reinterpret_cast<float4*>(smem + u * PU * 4);
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        d[i] = i < v ? __uint_as_float(s.w[i]) : 0.f;
        h[i] = __fmul_rn(h[i], q);
        if (i < v) acc = __fmaf_rn(__fmul_rn(d[i], g[i]), h[i], acc);
      }
#pragma unroll
      for (int i = 0; i < PU / 4; ++i) {
        sm[i] = make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
        float4 t = first ? make_float4(0.f, 0.f, 0.f, 0.f) : part[u * (PU / 4) + i];
        // columns past the end have d = 0 and are not read again
        t.x = __fmaf_rn(d[4 * i], h[4 * i], t.x);
        t.y = __fmaf_rn(d[4 * i + 1], h[4 * i + 1], t.y);
        t.z = __fmaf_rn(d[4 * i + 2], h[4 * i + 2], t.z);
        t.w = __fmaf_rn(d[4 * i + 3], h[4 * i + 3], t.w);
        part[u * (PU / 4) + i] = t;
      }
    }
    const float mean = block_sum(acc, s_part[flip]) / (float)hidden;
    for (size_t u = tid; u < units; u += blockDim.x) {
      const int v = a.vec ? PU : unit_valid<DT>(u, hidden);
      float h[PU], g[PU];
      code_floats<DT>(load_codes<DT>(crow, u, v, a.vec), pow2((int)__ldg(erow + u * PU / kCkptBlock) - 127), h);
      load_gamma<DT>(a.gamma, u, v, a.vec, g);
      const float* d = reinterpret_cast<const float*>(smem + u * PU * 4);
      Acc y;
#pragma unroll
      for (int i = 0; i < PU; ++i)
        y.w[i] = __float_as_uint(__fmul_rn(q, __fmaf_rn(-__fmul_rn(h[i], q), mean, __fmul_rn(d[i], g[i]))));
      const uint4 o = acc_narrow<DT>(y);
      if (a.vec) {
#pragma unroll
        for (int r = 0; r < N; ++r) st_stream(static_cast<char*>(a.out[r]) + row_off + u * 16, o);
      } else {
        *reinterpret_cast<uint4*>(smem + u * PU * 4) = o;
      }
    }
    if (!a.vec) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < N; ++r) store_row_any<DT>(static_cast<char*>(a.out[r]) + row_off, smem, PU * 4, hidden);
      __syncthreads();
    }
  }
}

// dgamma[c] = sum over the CTAs' partial rows, in order: 32 columns x 32
// strided row groups per CTA (LOOP: every gridDim-th 32 columns).
template <bool LOOP>
__global__ void __launch_bounds__(1024) dgamma_join_kernel(const float* part, int parts, size_t pitch, size_t hidden,
                                                           float* dgamma) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  pdl_wait();
  pdl_next();
  size_t c0 = (size_t)blockIdx.x * 32;
  do {
    const size_t c = c0 + lane;
    float v = 0.f;
    if (c < hidden) {
#pragma unroll 4
      for (int i = k; i < parts; i += 32) v += part[(size_t)i * pitch + c];
    }
    red[k][lane] = v;
    __syncthreads();
    // thread (k, lane) takes row group `lane` of column k: one warp a column
    float t = red[lane][k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0 && c0 + k < hidden) dgamma[c0 + k] = t;
    c0 += (size_t)gridDim.x * 32;
    if (LOOP) __syncthreads();  // red is free
  } while (LOOP && c0 < hidden);
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

constexpr int kN8SmemMax = 210 * 1024;
static size_t row_smem(size_t hidden) { return (hidden + 7) / 8 * 8 * sizeof(float); }
static bool fits_regs(int dt, bool vec, size_t hidden) {
  const size_t pu = dt == RRA_BFLOAT16 ? 8 : 4;
  return vec && hidden / pu <= kN8Regs / pu * kN8Threads;
}

template <int N, int DT, bool LOOP>
static cudaError_t save_go(Save8Args a, int grid, cudaStream_t s) {
  if (fits_regs(DT, a.vec, a.hidden)) return launch_pdl(save8_reg_kernel<N, DT, LOOP>, grid, kN8Threads, 0, s, a);
  const cudaError_t attr = raise_smem<save8_gen_kernel<N, DT, LOOP>>(kN8SmemMax);
  if (attr != cudaSuccess) return attr;
  size_t smem = row_smem(a.hidden);
  if (!a.vec && smem + smem / 4 <= kN8SmemMax) {
    a.stage_codes = 1;
    smem += smem / 4;
  }
  return launch_pdl(save8_gen_kernel<N, DT, LOOP>, grid, kN8Threads, smem, s, a);
}

// CTAs of the backward kernel: all resident, every CTA the same number of
// rows but for the last.
static int even_ctas(size_t rows, int most, int resident) {
  const size_t cap = most < resident ? most : resident;
  const size_t per = (rows + cap - 1) / cap;
  return (int)((rows + per - 1) / per);
}

template <int N, int DT>
static cudaError_t back_go(const Back8Args& a, int* ctas, cudaStream_t s) {
  if (fits_regs(DT, a.vec, a.hidden)) {
    *ctas = even_ctas(a.rows, *ctas, 2 * device_sms());
    return launch_pdl(back8_reg_kernel<N, DT>, *ctas, kN8Threads, 0, s, a);
  }
  const cudaError_t attr = raise_smem<back8_gen_kernel<N, DT>>(kN8SmemMax);
  if (attr != cudaSuccess) return attr;
  // as few trips over a row as kN8MaxThreads allow, all of them full
  const int units = (int)((a.hidden + 16 / Elem<DT>::kSize - 1) / (16 / Elem<DT>::kSize));
  const int trips = (units + kN8MaxThreads - 1) / kN8MaxThreads;
  const int threads = ((units + trips - 1) / trips + 31) / 32 * 32;
  int occ = 0;
  const cudaError_t err =
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, back8_gen_kernel<N, DT>, threads, row_smem(a.hidden));
  if (err != cudaSuccess) return err;
  *ctas = even_ctas(a.rows, *ctas, (occ > 0 ? occ : 1) * device_sms());
  return launch_pdl(back8_gen_kernel<N, DT>, *ctas, threads, row_smem(a.hidden), s, a);
}

template <int N>
static cudaError_t save_n(int dt, const Save8Args& a, cudaStream_t s) {
  const int grid = budget(a.rows);
  if ((size_t)grid < a.rows)
    return dt == RRA_FLOAT32 ? save_go<N, RRA_FLOAT32, true>(a, grid, s) : save_go<N, RRA_BFLOAT16, true>(a, grid, s);
  return dt == RRA_FLOAT32 ? save_go<N, RRA_FLOAT32, false>(a, grid, s) : save_go<N, RRA_BFLOAT16, false>(a, grid, s);
}

template <int N>
static cudaError_t back_n(int dt, const Back8Args& a, int* ctas, cudaStream_t s) {
  return dt == RRA_FLOAT32 ? back_go<N, RRA_FLOAT32>(a, ctas, s) : back_go<N, RRA_BFLOAT16>(a, ctas, s);
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
  a.vec = vec;
  switch (n) {
    case 1: return save_n<1>(dt, a, s);
    case 2: return save_n<2>(dt, a, s);
    case 3: return save_n<3>(dt, a, s);
    case 4: return save_n<4>(dt, a, s);
    case 5: return save_n<5>(dt, a, s);
    case 6: return save_n<6>(dt, a, s);
    case 7: return save_n<7>(dt, a, s);
    case 8: return save_n<8>(dt, a, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int DT, bool VEC>
static cudaError_t restore_go(const uint8_t* c, const uint8_t* e, const float* rstd, const void* gamma, void* out,
                              size_t rows, size_t hidden, int grid, cudaStream_t s) {
  if constexpr (!VEC) {
    const cudaError_t attr = raise_smem<restore8_kernel<DT, VEC>>(kN8SmemMax);
    if (attr != cudaSuccess) return attr;
  }
  return launch_pdl(restore8_kernel<DT, VEC>, grid, kN8Threads, VEC ? 0 : row_smem(hidden), s, c, e, rstd, gamma, out,
                    rows, hidden);
}

cudaError_t launch_norm_restore8(int dt, bool vec, const void* codes, const void* scales, const float* rstd,
                                 const void* gamma, void* out, size_t rows, size_t hidden, cudaStream_t s) {
  const size_t cap = max_ctas_cap() > 0 ? max_ctas_cap() : (size_t)device_sms() * 8;
  const int grid = (int)(rows < cap ? rows : cap);
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  const uint8_t* e = static_cast<const uint8_t*>(scales);
  if (dt == RRA_FLOAT32)
    return vec ? restore_go<RRA_FLOAT32, true>(c, e, rstd, gamma, out, rows, hidden, grid, s)
               : restore_go<RRA_FLOAT32, false>(c, e, rstd, gamma, out, rows, hidden, grid, s);
  return vec ? restore_go<RRA_BFLOAT16, true>(c, e, rstd, gamma, out, rows, hidden, grid, s)
             : restore_go<RRA_BFLOAT16, false>(c, e, rstd, gamma, out, rows, hidden, grid, s);
}

int norm_back8_ctas(size_t rows) {
  const size_t cap = 608;  // 4 per SM of 152
  return (int)(rows < cap ? rows : cap);
}

size_t norm_back8_pitch(size_t hidden) { return (hidden + 7) / 8 * 8; }

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
  a.pitch = norm_back8_pitch(hidden);
  a.rows = rows;
  a.hidden = hidden;
  a.vec = vec;
  int ctas = norm_back8_ctas(rows);
  if (max_ctas_cap() > 0 && max_ctas_cap() < ctas) ctas = max_ctas_cap();
  cudaError_t e;
  switch (n) {
    case 1: e = back_n<1>(dt, a, &ctas, s); break;
    case 2: e = back_n<2>(dt, a, &ctas, s); break;
    case 3: e = back_n<3>(dt, a, &ctas, s); break;
    case 4: e = back_n<4>(dt, a, &ctas, s); break;
    case 5: e = back_n<5>(dt, a, &ctas, s); break;
    case 6: e = back_n<6>(dt, a, &ctas, s); break;
    case 7: e = back_n<7>(dt, a, &ctas, s); break;
    case 8: e = back_n<8>(dt, a, &ctas, s); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  const size_t want = (hidden + 31) / 32;
  const int grid = budget(want);
  return launch_pdl((size_t)grid < want ? dgamma_join_kernel<true> : dgamma_join_kernel<false>, grid, 1024, 0, s, part,
                    ctas, a.pitch, hidden, dgamma);
}

}  // namespace rra
