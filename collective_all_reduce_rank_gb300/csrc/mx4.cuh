// mx4.cuh -- microscaled 4-bit floating point (MX4): 32 consecutive columns of
// a row share a power-of-two scale.
//
//   e = the smallest integer >= -127 with max |x| <= 6 * 2^e
//   code = e2m1(x * 2^-e): 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign, nearest, ties
//   to even; scale byte e + 127
//
// x * 2^-e is exact, so e2m1's rounding is the only one, and no value is
// clipped.  A block that holds an infinity or a NaN has no value to scale by:
// its scale byte is 255 (NaN) and its codes 0, so that the block, and a product
// it enters, reads as NaN.
//
// Layout, as the tensor cores read it.  Codes: rows of 16 bytes a block, the
// even column in a byte's low half.  Scales: tiles of 128 rows x 4 blocks, 512
// bytes each, the tiles of a row band side by side: a byte of (row, block) at
// row % 32 * 16 + row % 128 / 32 * 4 + block % 4 of its tile, which is the order
// in which tensor memory takes them (32 lanes of 4 words).
#pragma once

#include <cuda_fp4.h>

#include "rowio.cuh"

namespace rra {

constexpr int kMxBlock = 32;
constexpr uint32_t kMxNan = 255;

// Scale byte of a block whose largest |x| has these float32 bits.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax) {
  if (amax >= 0x7F800000u) return kMxNan;
  // (1 + m) 2^(E - 127) <= 1.5 * 2^2 * 2^e: e = E - 129 up to m = 0.5, else one more
  const int e = (int)(amax >> 23) - 2 + ((amax & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return (uint32_t)max(e, 0);
}

// 2^-e for a scale byte (e + 127) of mx_scale; 0 for the NaN block's codes.
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == kMxNan ? 0.f : __uint_as_float((254u - byte) << 23);
}

// 2^e of any scale byte; 2^-127 is below float32's normal range.
__device__ __forceinline__ float mx_power(uint32_t byte) {
  return byte == 0 ? __uint_as_float(0x00400000u)
                   : byte == kMxNan ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// Two codes as a byte, the first in the low half.
__device__ __forceinline__ uint32_t mx_code2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
}

__device__ __forceinline__ float2 mx_value2(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight scaled values as a word.  nan: the codes of a block without a scale
// (inf * 0 would make them the largest code).
__device__ __forceinline__ uint32_t mx_code8(const float* f, float inv, bool nan) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= mx_code2(f[2 * i] * inv, f[2 * i + 1] * inv) << (8 * i);
  return nan ? 0u : w;
}

__device__ __forceinline__ uint32_t mx_abs(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t mx_amax8(const float* f) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mx_abs(f[i]));
  return m;
}

// Byte offset of (row, block); `across`: tiles of a row band.
__host__ __device__ __forceinline__ size_t mx_scale_at(size_t row, size_t block, size_t across) {
  return (row / 128 * across + block / 4) * 512 + (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4;
}

// Eight columns of a row, float32: octet o, of which `valid` columns exist
// (zeros behind them).  vec: rows of whole aligned 16-byte units.
template <int DT>
__device__ __forceinline__ void load8(const char* row, size_t o, int valid, bool vec, float* f) {
  if constexpr (DT == RRA_BFLOAT16) {
    unit_floats<DT>(load_row<DT>(row, o, valid, vec), f);
  } else {
    unit_floats<DT>(load_row<DT>(row, 2 * o, min(valid, 4), vec), f);
    if (valid > 4) {
      unit_floats<DT>(load_row<DT>(row, 2 * o + 1, valid - 4, vec), f + 4);
    } else {
#pragma unroll
      for (int i = 4; i < 8; ++i) f[i] = 0.f;
    }
  }
}

// The same columns stored, rounded to DT once.
template <int DT>
__device__ __forceinline__ void store8(char* row, size_t o, int valid, bool vec, const float* f) {
  Acc a;
#pragma unroll
  for (int i = 0; i < 8; ++i) a.w[i] = __float_as_uint(f[i]);
  if constexpr (DT == RRA_BFLOAT16) {
    const uint4 v = acc_narrow<DT>(a);
    if (vec)
      st_stream(row + o * 16, v);
    else
      st_partial<DT>(row + o * 16, v, valid);
  } else {
    const uint4 v0 = make_uint4(a.w[0], a.w[1], a.w[2], a.w[3]), v1 = make_uint4(a.w[4], a.w[5], a.w[6], a.w[7]);
    if (vec) {
      st_stream(row + o * 32, v0);
      if (valid > 4) st_stream(row + o * 32 + 16, v1);
    } else {
      st_partial<DT>(row + o * 32, v0, min(valid, 4));
      if (valid > 4) st_partial<DT>(row + o * 32 + 16, v1, valid - 4);
    }
  }
}

// Columns of octet o that a row of `cols` has.
__device__ __forceinline__ int octet_valid(size_t o, size_t cols) {
  return o * 8 + 8 <= cols ? 8 : (o * 8 < cols ? (int)(cols - o * 8) : 0);
}

// Quantise a block held by four neighbouring lanes, eight columns each, and
// store it: the codes, and with the fourth block of a tile's row (the first of
// 16 lanes) that row's scale word.  All 32 lanes call this, lane l with an
// octet o of which o % 16 == l % 16; octets behind the row's last block (up to
// the tile's fourth) have f = 0 and store their scale byte 0, which a product
// may read, but no codes.
__device__ __forceinline__ void mx_put8(const float* f, uint8_t* codes, uint8_t* scales, size_t row, size_t o,
                                        size_t octets, size_t across, bool live) {
  uint32_t m = mx_amax8(f);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t byte = mx_scale(m);
  const uint32_t w = mx_code8(f, mx_inverse(byte), byte == kMxNan);
  uint32_t s = byte << (8 * ((threadIdx.x >> 2) & 3));
  s |= __shfl_xor_sync(0xffffffffu, s, 4);
  s |= __shfl_xor_sync(0xffffffffu, s, 8);
  if (!live) return;
  if (o < octets) *reinterpret_cast<uint32_t*>(codes + (row * octets + o) * 4) = w;
  if ((threadIdx.x & 15) == 0 && o < across * 16)
    *reinterpret_cast<uint32_t*>(scales + mx_scale_at(row, o / 4, across)) = s;
}

}  // namespace rra
