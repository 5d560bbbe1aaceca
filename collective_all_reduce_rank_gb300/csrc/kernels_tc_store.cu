// kernels_tc_store.cu -- the two gradient products of the training operators
// (input gradient dx = sum_r D_r W_r, weight gradient dW_r = D_r^T x) and the
// small row-wise kernels around the products.
//
// The input gradient walks the shards of all virtual ranks as segments of
// one K axis, so the sum over ranks that a tensor-parallel step leaves to an
// all-reduce is the accumulation in tensor memory, in float32.
#include "tc_epilogue.cuh"

namespace rra {

template <bool F32>
struct EpiStore {
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row, int half, uint32_t addr) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 256 + half * 128;
    const long long off = (long long)row * g.ld + c0;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      const int valid = g.N - c0 - c;
      if (valid <= 0) break;
      float v[32];
      tc_ld32(addr + half * 128 + c, v);
      tc_ld_wait();
      if (row >= g.M) continue;
      if constexpr (F32) {
        float* o = static_cast<float*>(g.out) + x.split * p.split_stride + off + c;
        if (g.vec && valid >= 32) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float4 w = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            if (p.accumulate) {
              const float4 q = *reinterpret_cast<const float4*>(o + j);
              w = make_float4(q.x + w.x, q.y + w.y, q.z + w.z, q.w + w.w);
            }
            *reinterpret_cast<float4*>(o + j) = w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < valid) o[j] = p.accumulate ? o[j] + v[j] : v[j];
        }
      } else {
        tc_store_bf16(static_cast<__nv_bfloat16*>(g.out) + off + c, v, valid, g.vec, false);
      }
    }
  }
};

cudaError_t launch_tc_input_grad(const TcArgs& p, bool f32, cudaStream_t s, int* grid) {
  return f32 ? tc_launch<false, true, EpiStore<true>>(p, s, grid) : tc_launch<false, true, EpiStore<false>>(p, s, grid);
}

cudaError_t launch_tc_weight_grad(const TcArgs& p, cudaStream_t s, int* grid) {
  return tc_launch<true, true, EpiStore<false>>(p, s, grid);
}

// ---------------------------------------------------------------------------

constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads) join_slots_kernel(const float* slots, int n, long long stride,
                                                                 __nv_bfloat16* out, long long count) {
  const long long step = (long long)gridDim.x * kRowThreads;
  for (long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x; i < count; i += step) {
    float v = slots[i];
    for (int k = 1; k < n; ++k) v += slots[k * stride + i];
    out[i] = __float2bfloat16_rn(v);
  }
}

cudaError_t launch_join_slots(const float* slots, int n, long long stride, void* out, long long count,
                              cudaStream_t s) {
  const int cap = max_ctas_cap() > 0 ? max_ctas_cap() : device_sms() * 8;
  const long long want = (count + kRowThreads - 1) / kRowThreads;
  join_slots_kernel<<<(int)(want < cap ? want : cap), kRowThreads, 0, s>>>(slots, n, stride,
                                                                          static_cast<__nv_bfloat16*>(out), count);
  return cudaGetLastError();
}

__global__ void __launch_bounds__(kRowThreads) pad_rows_kernel(const uint16_t* src, uint16_t* dst, long long rows,
                                                               long long cols, long long ld) {
  for (long long r = blockIdx.x; r < rows; r += gridDim.x)
    for (long long c = threadIdx.x; c < cols; c += kRowThreads) dst[r * ld + c] = __ldg(src + r * cols + c);
}

cudaError_t launch_pad_rows(const void* src, void* dst, long long rows, long long cols, long long ld,
                            cudaStream_t s) {
  const int cap = max_ctas_cap() > 0 ? max_ctas_cap() : device_sms() * 8;
  pad_rows_kernel<<<(int)(rows < cap ? rows : cap), kRowThreads, 0, s>>>(
      static_cast<const uint16_t*>(src), static_cast<uint16_t*>(dst), rows, cols, ld);
  return cudaGetLastError();
}

}  // namespace rra
