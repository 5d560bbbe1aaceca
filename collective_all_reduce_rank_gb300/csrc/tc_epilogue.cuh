// tc_epilogue.cuh -- row pieces between registers and memory for the
// epilogues of tc_gemm.cuh: one lane holds 32 consecutive columns of a row
// in float32.
#pragma once

#include "tc_gemm.cuh"

namespace rra {

__device__ __forceinline__ uint32_t tc_pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// What bfloat16 leaves of v (nothing of what it makes infinite).
__device__ __forceinline__ float tc_left(float v) {
  const float held = __bfloat162float(__float2bfloat16_rn(v));
  return fabsf(held) < INFINITY ? v - held : 0.f;
}

// Stores go through a warp's staging buffer: a lane holds 128 bytes of one
// row (64 bfloat16 or 32 float32), which it writes as 16-byte chunks in a
// swizzled order (chunk c of row r at c ^ (r & 7): no bank conflicts either
// way), and the warp then stores whole rows, 8 lanes a row, so that every
// store covers full 128-byte lines.  Straight from registers a warp's store
// touched 32 rows: rows of 515 bfloat16 (no 16-byte stores) took 268 us for
// the 333 x 515 x 50021 weight gradient.
__device__ __forceinline__ void tc_stage_bf16(uint8_t* buf, const float* v, int first_chunk) {
  const int r = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(buf + r * 128 + (((first_chunk + c) ^ (r & 7)) << 4)) =
        make_uint4(tc_pack2(v[8 * c], v[8 * c + 1]), tc_pack2(v[8 * c + 2], v[8 * c + 3]),
                   tc_pack2(v[8 * c + 4], v[8 * c + 5]), tc_pack2(v[8 * c + 6], v[8 * c + 7]));
}

// What bfloat16 leaves of 32 values, packed, and such pairs as chunks of a row.
__device__ __forceinline__ void tc_left2(const float* v, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) w[j / 2] = tc_pack2(tc_left(v[j]), tc_left(v[j + 1]));
}

__device__ __forceinline__ void tc_stage_packed(uint8_t* buf, const uint32_t* w, int first_chunk) {
  const int r = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(buf + r * 128 + (((first_chunk + c) ^ (r & 7)) << 4)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

// Store `rows` rows (clipped to [0, 32]) of `valid` bfloat16 (clipped to [0,
// 64]) from the staging buffer to dst, rows ld elements apart.  vec: dst
// rows start on 16 bytes; `pad`: they have room up to the next multiple of
// 8, so a partial chunk is stored whole.
__device__ __forceinline__ void tc_flush_bf16(const uint8_t* buf, __nv_bfloat16* dst, long long ld, int rows, int valid,
                                              bool vec, bool pad) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (vec) {
    const int c = lane & 7;
    const int left = valid - 8 * c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      if (r >= rows || left <= 0) continue;
      const uint4 u = *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
      __nv_bfloat16* o = dst + r * ld + 8 * c;
      if (left >= 8 || pad) {
        *reinterpret_cast<uint4*>(o) = u;
      } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        for (int j = 0; j < left; ++j)
          reinterpret_cast<uint16_t*>(o)[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      }
    }
  } else {
    // rows of any alignment: lane l holds elements 2l and 2l + 1 as one
    // word; in a row that starts between two words of memory every lane
    // takes its second element and its neighbour's first instead
    const uint8_t* src = buf + ((lane & 3) << 2);
    uint16_t* o = reinterpret_cast<uint16_t*>(dst);
    if (rows >= 32 && valid >= 64) {
      // whole block: 8 rows at a time, so that the shared-memory reads, the
      // shuffles and the stores of different rows overlap
      const bool edge = lane == 0 || lane == 31;
#pragma unroll 1
      for (int r0 = 0; r0 < 32; r0 += 8) {
        uint32_t w[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = *reinterpret_cast<const uint32_t*>(src + (r0 + i) * 128 + (((lane >> 2) ^ i) << 4));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __funnelshift_r(w[i], __shfl_down_sync(0xffffffffu, w[i], 1), 16);
#pragma unroll
        for (int i = 0; i < 8; ++i, o += ld) {
          // stores under predicates, not branches, so that the rows stay in flight together
          const uint32_t odd = ((uint32_t)(uintptr_t)o >> 1) & 1;
          asm volatile(
              "{\n.reg .pred p, q;\n"
              "setp.ne.u32 p, %2, 0;\n@p st.global.u32 [%0], %1;\n"
              "setp.ne.u32 q, %5, 0;\n@q st.global.u16 [%3], %4;\n}\n" ::"l"(o + 2 * lane + odd),
              "r"(odd ? v[i] : w[i]), "r"((uint32_t)(lane < 31 || !odd)), "l"(o + (lane == 0 ? 0 : 63)),
              "h"((uint16_t)(lane == 0 ? w[i] : w[i] >> 16)), "r"((uint32_t)(odd && edge))
              : "memory");
        }
      }
    } else {
      const int top = rows < 32 ? rows : 32;
      const int j0 = 2 * lane;
      for (int r = 0; r < top; ++r, o += ld) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(src + r * 128 + (((lane >> 2) ^ (r & 7)) << 4));
        const uint32_t next = __shfl_down_sync(0xffffffffu, w, 1);
        const int odd = (int)(((uintptr_t)o >> 1) & 1);
        const int j = j0 + odd;
        const uint32_t v = odd ? __funnelshift_r(w, next, 16) : w;
        if (j + 1 < valid && j < 63)
          *reinterpret_cast<uint32_t*>(o + j) = v;
        else if (j < valid)
          o[j] = (uint16_t)v;
        if (odd && lane == 0 && valid > 0) o[0] = (uint16_t)w;
      }
    }
  }
  __syncwarp();
}

// Rows of 32 + 32 bfloat16 to two destinations with 16-byte rows padded to
// whole chunks.
__device__ __forceinline__ void tc_flush_pair(const uint8_t* buf, __nv_bfloat16* d0, __nv_bfloat16* d1, long long ld,
                                              int rows, int valid) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  __nv_bfloat16* dst = c < 4 ? d0 : d1;
  __syncwarp();
  if (8 * (c & 3) < valid) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      if (r < rows)
        *reinterpret_cast<uint4*>(dst + r * ld + 8 * (c & 3)) =
            *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
    }
  }
  __syncwarp();
}

// The same for 32 float32 a row (vec: 16-byte rows); add: dst += row.
__device__ __forceinline__ void tc_store_f32(uint8_t* buf, const float* v, float* dst, long long ld, int rows,
                                             int valid, bool vec, bool add) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
  if (vec && valid >= 32) {
    const int c = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      if (r >= rows) continue;
      float4 u = *reinterpret_cast<const float4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
      float4* o = reinterpret_cast<float4*>(dst + r * ld + 4 * c);
      if (add) {
        const float4 q = *o;
        u = make_float4(q.x + u.x, q.y + u.y, q.z + u.z, q.w + u.w);
      }
      *o = u;
    }
  } else {
    const float* e = reinterpret_cast<const float*>(buf);
    for (int r = 0; r < rows && r < 32; ++r) {
      float* o = dst + r * ld + lane;
      if (lane < valid) {
        const float u = e[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)];
        *o = add ? *o + u : u;
      }
    }
  }
  __syncwarp();
}

// Load 32 rows of 32 bfloat16 (zeros outside `rows` x `valid`), each lane its
// row's, through the staging buffer so that the loads cover whole rows.
__device__ __forceinline__ void tc_load_bf16(uint8_t* buf, const __nv_bfloat16* src, long long ld, int rows, int valid,
                                             bool vec, float* v) {
  const int lane = threadIdx.x & 31;
  if (vec && valid >= 32) {
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2);
      u[i] = r < rows ? __ldg(reinterpret_cast<const uint4*>(src + r * ld + 8 * (lane & 3))) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2);
      *reinterpret_cast<uint4*>(buf + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)) = u[i];
    }
  } else {
    const int c = 2 * (lane & 15);
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int r = 2 * i + (lane >> 4);
      const uint16_t* p = reinterpret_cast<const uint16_t*>(src) + r * ld + c;
      const uint32_t a = r < rows && c < valid ? __ldg(p) : 0u;
      const uint32_t b = r < rows && c + 1 < valid ? __ldg(p + 1) : 0u;
      *reinterpret_cast<uint32_t*>(buf + r * 64 + (((c >> 3) ^ ((r >> 1) & 3)) << 4) + 2 * (c & 7)) = a | (b << 16);
    }
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 q = *reinterpret_cast<const uint4*>(buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * c + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * c + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  __syncwarp();
}

}  // namespace rra
