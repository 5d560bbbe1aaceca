// rowio.cuh -- 16-byte units of rows that may start on any element.
#pragma once

#include "common.cuh"

namespace rra {

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

}  // namespace rra
