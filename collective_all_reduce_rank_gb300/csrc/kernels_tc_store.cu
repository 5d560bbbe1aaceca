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
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row0, int half, uint32_t addr,
                                             uint8_t* buf) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 256 + half * 128;
    const int rows = g.M - row0;
    const long long off = (long long)row0 * g.ld + c0;
    constexpr int STEP = F32 ? 32 : 64;
#pragma unroll 1
    for (int c = 0; c < 128; c += STEP) {
      const int valid = g.N - c0 - c;
      if (valid <= 0) break;
      float v[32];
      tc_ld32(addr + half * 128 + c, v);
      if constexpr (F32) {
        tc_ld_wait();
        float* o = static_cast<float*>(g.out) + x.split * p.split_stride + off + c;
        tc_store_f32(buf, v, o, g.ld, rows, valid, g.vec, p.accumulate);
      } else {
        float w[32];
        tc_ld32(addr + half * 128 + c + 32, w);
        tc_ld_wait();
        tc_stage_bf16(buf, v, 0);
        tc_stage_bf16(buf, w, 4);
        tc_flush_bf16(buf, static_cast<__nv_bfloat16*>(g.out) + off + c, g.ld, rows, valid, g.vec, false);
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

// out[r][c] = bfloat16(sum over the slots), slots' rows ld (a multiple of 8)
// elements apart; a thread takes 8 columns, a CTA whole rows.
__global__ void __launch_bounds__(kRowThreads)
    join_slots_kernel(const float* slots, int n, long long stride, int ld, __nv_bfloat16* out, int rows, int cols,
                      int vec) {
  pdl_wait();
  pdl_next();
  const int units = ld / 8;
  const long long total = (long long)rows * units, step = (long long)gridDim.x * kRowThreads;
  for (long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x; i < total; i += step) {
    const int r = total <= 0xFFFFFFFFll ? (int)((uint32_t)i / (uint32_t)units) : (int)(i / units);
    const int c = (int)(i - (long long)r * units) * 8;
    const float4* p = reinterpret_cast<const float4*>(slots + (long long)r * ld + c);
    float4 a = __ldcs(p), b = __ldcs(p + 1);
    for (int k = 1; k < n; ++k) {
      const float4* q = reinterpret_cast<const float4*>(slots + k * stride + (long long)r * ld + c);
      const float4 x = __ldcs(q), y = __ldcs(q + 1);
      a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
      b = make_float4(b.x + y.x, b.y + y.y, b.z + y.z, b.w + y.w);
    }
    __nv_bfloat16* o = out + (long long)r * cols + c;
    const uint32_t w[4] = {tc_pack2(a.x, a.y), tc_pack2(a.z, a.w), tc_pack2(b.x, b.y), tc_pack2(b.z, b.w)};
    if (vec && c + 8 <= cols) {
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) reinterpret_cast<uint16_t*>(o)[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

cudaError_t launch_join_slots(const float* slots, int n, long long stride, int ld, void* out, int rows, int cols,
                              cudaStream_t s) {
  const long long cap = max_ctas_cap() > 0 ? max_ctas_cap() : device_sms() * 8;
  const long long want = ((long long)rows * (ld / 8) + kRowThreads - 1) / kRowThreads;
  const int vec = cols % 8 == 0 && ((uintptr_t)out & 15) == 0;
  return launch_pdl(join_slots_kernel, (int)(want < cap ? want : cap), kRowThreads, 0, s, slots, n, stride, ld,
                    static_cast<__nv_bfloat16*>(out), rows, cols, vec);
}

// Rows of up to 17 matrices to padded rows (16-byte units), one launch: a
// thread writes one unit of a destination row.
__global__ void __launch_bounds__(kRowThreads) pad_rows_kernel(const __grid_constant__ PadArgs a) {
  pdl_wait();
  pdl_next();
  const long long step = (long long)gridDim.x * kRowThreads;
  int m = 0;
  for (long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x; i < a.first[a.n]; i += step) {
    while (i >= a.first[m + 1]) ++m;
    const long long u = i - a.first[m];
    const long long row = u < 0xFFFFFFFFll ? (long long)((uint32_t)u / (uint32_t)a.units) : u / a.units;
    const int c = (int)(u - row * a.units) * 8;
    const uint16_t* src = static_cast<const uint16_t*>(a.src[m]) + row * a.cols + c;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = c + 2 * j < a.cols ? __ldg(src + 2 * j) : 0u;
      const uint32_t hi = c + 2 * j + 1 < a.cols ? __ldg(src + 2 * j + 1) : 0u;
      w[j] = lo | (hi << 16);
    }
    reinterpret_cast<uint4*>(a.dst[m])[u] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

cudaError_t launch_pad_rows(const PadArgs& a, cudaStream_t s) {
  const long long want = (a.first[a.n] + kRowThreads - 1) / kRowThreads;
  if (want == 0) return cudaSuccess;
  const long long cap = max_ctas_cap() > 0 ? max_ctas_cap() : device_sms() * 8;
  return launch_pdl(pad_rows_kernel, (int)(want < cap ? want : cap), kRowThreads, 0, s, a);
}

}  // namespace rra
