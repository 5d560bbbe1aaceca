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

#include <cuda_fp16.h>

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

// Eight values as a word of codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t mx_pack8(const float* f) {
  uint32_t w;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

// One code, in the lowest four bits.
__device__ __forceinline__ uint32_t mx_code(float x) {
  uint32_t w;
  asm("{\n.reg .b8 a, z;\ncvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\nmov.b32 %0, {a, a, a, a};\n}\n"
      : "=r"(w)
      : "f"(x), "f"(0.f));
  return w & 15u;
}

// Eight scaled values as a word.  nan: the codes of a block without a scale
// (inf * 0 would make them the largest code).
__device__ __forceinline__ uint32_t mx_code8(const float* f, float inv, bool nan) {
  float g[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = f[i] * inv;
  return nan ? 0u : mx_pack8(g);
}

// The same of a unit of bfloat16: the multiplication widens.  -0 is added so
// that zeros keep their sign.
__device__ __forceinline__ uint32_t mx_code8(const uint4& x, uint32_t byte) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const uint16_t inv = (uint16_t)(byte == kMxNan ? 0u : (254u - byte) << 7);
  float g[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\n"
        "fma.rn.f32.bf16 %0, l, %3, %4;\nfma.rn.f32.bf16 %1, h, %3, %4;\n}"
        : "=f"(g[2 * i]), "=f"(g[2 * i + 1])
        : "r"(w[i]), "h"(inv), "f"(-0.f));
  return byte == kMxNan ? 0u : mx_pack8(g);
}

// The values of a word of codes times a power of two, exactly.
__device__ __forceinline__ void mx_value8(uint32_t w, float power, float* f) {
  uint32_t h[4];
  asm("{\n.reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = v.x * power;
    f[2 * i + 1] = v.y * power;
  }
}

// The value of the code in the lowest four bits.
__device__ __forceinline__ float mx_value(uint32_t code) {
  const uint32_t m = code & 7u;
  // the code's bits as those of a float32 2^126 times as small: e and m in place, 0.5 a subnormal
  const float v = __uint_as_float(m << 22) * __uint_as_float(0x7E800000u);
  return code & 8u ? -v : v;
}

__device__ __forceinline__ uint32_t mx_abs(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Float32 bits of the largest |x| of a unit of bfloat16.
__device__ __forceinline__ uint32_t mx_amax_bf16(const uint4& x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                              __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}

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

// A row of an MX4 matrix being written or read: where its codes start, and the
// scale bytes of its first tile (tile t's are 512 t further, in 32 bits:
// mx_from).
struct MxRow {
  uint32_t octets;  // words of codes
  uint32_t ends;    // octets up to the last tile's end
  uint32_t* codes;
  uint8_t* scales;
};

__device__ __forceinline__ MxRow mx_row(const void* codes, const void* scales, size_t row, size_t cols) {
  const size_t across = (cols + 127) / 128, octets = (cols + 31) / 32 * 4;
  return {(uint32_t)octets, (uint32_t)(across * 16),
          const_cast<uint32_t*>(static_cast<const uint32_t*>(codes)) + row * octets,
          const_cast<uint8_t*>(static_cast<const uint8_t*>(scales)) + row / 128 * across * 512 +
              ((uint32_t)row % 32 * 16 + (uint32_t)row % 128 / 32 * 4)};
}

// The row for octets near `o`: where 512 t passes 32 bits (column 2^30) the
// scales start a multiple of 2^32 further.  (16384 x 5120: with 512 t in 64 bits
// bfloat16 quantised in 41.1 us and float32 read back in 86, this way 39.4 and
// 82, as without either.)
__device__ __forceinline__ MxRow mx_from(MxRow r, uint32_t o) {
  r.scales += (size_t)(o >> 27) << 32;
  return r;
}

// Quantise a block held by four neighbouring lanes, eight columns each (m: bits
// of their largest value, code: their codes under a scale), and store it: the codes, and with the fourth block of a
// tile's row (the first of 16 lanes) that row's scale word.  All 32 lanes call
// this, lane l with an octet o of which o % 16 == l % 16; octets behind the
// row's last block (up to the tile's fourth) have f = 0 and store their scale
// byte 0, which a product may read, but no codes.
template <class Code>
__device__ __forceinline__ void mx_put8(uint32_t m, const MxRow& r, uint32_t o, Code code) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t byte = mx_scale(m);
  uint32_t s = byte << (8 * ((threadIdx.x >> 2) & 3));
  s |= __shfl_xor_sync(0xffffffffu, s, 4);
  s |= __shfl_xor_sync(0xffffffffu, s, 8);
  if (o < r.octets) r.codes[o] = code(byte);
  if ((threadIdx.x & 15) == 0 && o < r.ends) *reinterpret_cast<uint32_t*>(r.scales + (o / 16) * 512) = s;
}

__device__ __forceinline__ void mx_put8(const float* f, const MxRow& r, uint32_t o) {
  mx_put8(mx_amax8(f), r, o, [&](uint32_t byte) { return mx_code8(f, mx_inverse(byte), byte == kMxNan); });
}

__device__ __forceinline__ void mx_put8(const uint4& x, const MxRow& r, uint32_t o) {
  mx_put8(mx_amax_bf16(x), r, o, [&](uint32_t byte) { return mx_code8(x, byte); });
}

}  // namespace rra
