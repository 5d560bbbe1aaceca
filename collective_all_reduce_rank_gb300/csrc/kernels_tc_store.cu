// kernels_tc_store.cu -- the two gradient products of the training operators
// (input gradient dx = sum_r D_r W_r, weight gradient dW_r = D_r^T x) and the
// small row-wise kernels around the products.
//
// The input gradient walks the shards of all virtual ranks as segments of
// one K axis, so the sum over ranks that a tensor-parallel step leaves to an
// all-reduce is the accumulation in tensor memory, in float32.
//
// Measured (4096 tokens x 5120, 4 shards of 3456; one GB300): dx 0.59 ms, dW
// 0.61 ms for 1.16 TFLOP each, 1.97 and 1.92 PFLOP/s.  A weight gradient of
// few tokens is bound by writing it: rows of 16-byte units take full-line
// stores (333 tokens x 512 x 50021: 26 us), rows of any alignment 4-byte
// stores of a shifted row (x 515: 40 us).
#include "tc_epilogue.cuh"

namespace rra {

template <bool F32>
struct EpiStore {
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row0, int half, uint32_t addr,
                                             uint8_t* buf) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 256 + half * 128;
    const int rows = g.M - row0;
    const bool part = x.slot >= 0 && p.splits > 1;
    const int row = row0 + (threadIdx.x & 31);
    const float scale = p.row_scale && row < g.M ? p.row_scale[(long long)row * 4] : 1.f;
    if (F32 || part) {
      // float32 rows of the output, or the tile's own slot
      const long long ld = part ? 256 : g.ld;
      float* o = part ? p.slots + (long long)x.slot * 65536 + (row0 - x.m * 256) * 256 + half * 128
                      : static_cast<float*>(g.out) + (long long)row0 * g.ld + c0;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        const int valid = g.N - c0 - c;
        if (valid <= 0) break;
        float v[32];
        tc_ld32(addr + half * 128 + c, v);
        tc_ld_ready(v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= scale;
        tc_store_f32(buf, v, o + c, ld, rows, part ? 32 : valid, part || g.vec, p.accumulate);
      }
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g.out) + (long long)row0 * g.ld + c0;
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        const int valid = g.N - c0 - c;
        if (valid <= 0) break;
        float v[32], w[32];
        tc_ld32(addr + half * 128 + c, v);
        tc_ld32(addr + half * 128 + c + 32, w);
        tc_ld_ready(v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= scale;
        tc_stage_bf16(buf, v, 0);
        tc_ld_ready(w);
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] *= scale;
        tc_stage_bf16(buf, w, 4);
        tc_flush_bf16(buf, o + c, g.ld, rows, valid, g.vec, false);
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

// One CTA per 8 rows of a tile; a thread takes 8 columns of one.
__global__ void __launch_bounds__(kRowThreads) join_tiles_kernel(const __grid_constant__ JoinTiles j, int first) {
  pdl_wait();
  pdl_next();
  const int tile = first + blockIdx.x / 32, slab = blockIdx.x % 32;
  int m, n;
  tc_walk(tile, j.mt, j.nt, m, n);
  const bool vec = j.cols % 8 == 0 && ((uintptr_t)j.out & 15) == 0;
  const int lr = slab * 8 + (threadIdx.x >> 5), lc = (threadIdx.x & 31) * 8;
  const int r = m * 256 + lr, c = n * 256 + lc;
  if (r < j.rows && c < j.cols) {
    float4 a, b;
    if (tile < j.full || j.splits == 1) {
      const float4* q = reinterpret_cast<const float4*>(j.acc + (long long)r * j.ld + c);
      a = __ldcs(q);
      b = __ldcs(q + 1);
    } else {
      const float* q = j.slots + (long long)(tile - j.full) * j.splits * 65536 + lr * 256 + lc;
      a = __ldcs(reinterpret_cast<const float4*>(q));
      b = __ldcs(reinterpret_cast<const float4*>(q) + 1);
#pragma unroll 4
      for (int k = 1; k < j.splits; ++k) {
        const float4* z = reinterpret_cast<const float4*>(q + k * 65536);
        const float4 x = __ldcs(z), y = __ldcs(z + 1);
        a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
        b = make_float4(b.x + y.x, b.y + y.y, b.z + y.z, b.w + y.w);
      }
    }
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(j.out) + (long long)r * j.cols + c;
    const uint32_t w[4] = {tc_pack2(a.x, a.y), tc_pack2(a.z, a.w), tc_pack2(b.x, b.y), tc_pack2(b.z, b.w)};
    if (vec) {
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < j.cols) reinterpret_cast<uint16_t*>(o)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
  }
}

cudaError_t launch_join_tiles(const JoinTiles& j, cudaStream_t s) {
  // without `acc` the whole tiles are in the output already
  const int first = j.acc ? 0 : j.full, tiles = j.mt * j.nt;
  if (first >= tiles || (!j.acc && j.splits == 1)) return cudaSuccess;
  return launch_pdl(join_tiles_kernel, (tiles - first) * 32, kRowThreads, 0, s, j, first);
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
