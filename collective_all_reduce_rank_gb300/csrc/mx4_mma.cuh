// mx4_mma.cuh -- PTX of the block-scaled products: scales into tensor memory,
// the product itself.  Helpers of tc_gemm.cuh (barriers, waits, TMA loads of a
// pair of CTAs, accumulator reads) are used as they are there.
#pragma once

#include "mx4.cuh"
#include "serve_host.h"
#include "tc_epilogue.cuh"

namespace rra {

// Instruction descriptor: e2m1 operands, both K-major, E8M0 scales, M x N; the
// scale ids say which two of a word's four scales a 64-deep product takes.
__host__ __device__ constexpr uint32_t mx4_idesc(uint32_t m, uint32_t n) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t mx4_idesc_scales(uint32_t id) { return (id << 4) | (id << 29); }

// One lane of the warp, the same each time.
__device__ __forceinline__ bool mx4_elect() {
  uint32_t is;
  __syncwarp();
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(is));
  return is != 0;
}

// Shared-memory descriptor of a tile of scales: 32 rows of 16 bytes, no
// swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t mx4_scale_desc(uint32_t addr) {
  return ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46) | (uint64_t)((addr & 0x3FFFF) >> 4);
}

// A tile of scales (512 bytes) to four columns of tensor memory, once for each
// quarter of the lanes.  It runs in order with the products around it.
__device__ __forceinline__ void mx4_put_scales(uint32_t taddr, uint32_t addr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(mx4_scale_desc(addr)) : "memory");
}

// TMA tile load into this CTA that counts on its own barrier.
__device__ __forceinline__ void mx4_load(const CUtensorMap* map, uint32_t dst, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// 32 lanes x 8 words to tensor memory.
__device__ __forceinline__ void mx4_st8(uint32_t taddr, const uint4& a, const uint4& b) {
  __syncwarp();
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

__device__ __forceinline__ void mx4_st_wait() {
  __syncwarp();
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <bool PAIR>
__device__ __forceinline__ void mx4_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
        : "memory");
}

// 32 columns of one row of a gated block's activations, quantised and stored.
// `valid`: columns the row has from here on (0: none, the scale byte 0 alone).
__device__ __forceinline__ void mx4_put_row(float* v, int valid, uint8_t* codes, uint8_t* scale) {
  if (valid < 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j >= valid) v[j] = 0.f;
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = max(m, mx_abs(v[j]));
  const uint32_t byte = mx_scale(m);
  const float inv = mx_inverse(byte);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = mx_code8(v + 8 * q, inv, byte == kMxNan);
  if (valid > 0) *reinterpret_cast<uint4*>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
  *scale = (uint8_t)byte;
}

}  // namespace rra
