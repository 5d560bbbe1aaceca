// tc_epilogue.cuh -- row pieces between registers and memory for the
// epilogues of tc_gemm.cuh: one thread holds 32 consecutive columns of a
// row in float32.
#pragma once

#include "tc_gemm.cuh"

namespace rra {

__device__ __forceinline__ uint32_t tc_pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Store the first `valid` (clipped to [0, 32]) of 32 values as bfloat16.
// vec: 16-byte stores for whole groups of 8; `pad`: the row has room up to
// the next multiple of 8, so a partial group is stored whole.
__device__ __forceinline__ void tc_store_bf16(__nv_bfloat16* dst, const float* v, int valid, bool vec, bool pad) {
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    if (vec && (c + 8 <= valid || (pad && c < valid))) {
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(tc_pack2(v[c], v[c + 1]), tc_pack2(v[c + 2], v[c + 3]),
                                                      tc_pack2(v[c + 4], v[c + 5]), tc_pack2(v[c + 6], v[c + 7]));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < valid) dst[c + j] = __float2bfloat16_rn(v[c + j]);
    }
  }
}

// Load 32 bfloat16 (zeros from `valid` on).
__device__ __forceinline__ void tc_load_bf16(const __nv_bfloat16* src, float* v, int valid, bool vec) {
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    if (vec && c + 8 <= valid) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + c));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[c + 2 * j] = __uint_as_float(w[j] << 16);
        v[c + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c + j] = c + j < valid ? __bfloat162float(src[c + j]) : 0.f;
    }
  }
}

}  // namespace rra
