// kernels_tc_store.cu -- the two gradient products of the training operators
// (input gradient dx = sum_r D_r W_r, weight gradient dW_r = D_r^T x) and the
// small row-wise kernels around the products.
//
// The input gradient walks the shards of all virtual ranks as segments of
// one K axis, so the sum over ranks that a tensor-parallel step leaves to an
// all-reduce is the accumulation in tensor memory, in float32.
//
// Measured (4096 tokens x 5120, 4 shards of 3456; one GB300, a launch alone):
// dx 0.59 ms, dW 0.61 ms for 1.16 TFLOP each, 1.97 and 1.92 PFLOP/s; call after
// call the power limit makes them 15% longer.  A weight gradient of few tokens
// is bound by writing it: rows of 16-byte units take full-line stores (333
// tokens x 512 x 50021: 26 us), rows of any alignment 4-byte stores of a shifted
// row (x 515: 40 us, 50 with the targets' additions).
#include "tc_epilogue.cuh"

namespace rra {

// v[j] += f * row[c + j] for 32 columns (row 16-byte aligned, ld elements).
__device__ __forceinline__ void fix_add(float* v, float f, const __nv_bfloat16* row, int c, long long ld) {
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    if (c + k + 8 > ld) break;
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + c + k));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[k + 2 * j] = fmaf(f, __uint_as_float(w[j] << 16), v[k + 2 * j]);
      v[k + 2 * j + 1] = fmaf(f, __uint_as_float(w[j] & 0xFFFF0000u), v[k + 2 * j + 1]);
    }
  }
}

// The additions of TcFix to a warp's rows of a tile (row0 + lane of the
// group), from what was asked for a tile ahead.
struct FixState {
  int at, count;             // kind 2: the tokens whose targets are among the rows
  int owner, token;          // lane i: the i-th of them (of 32 at a time)
  float lo;                  // and its factor
  uint2 held[2];             // of the first two: columns 4 lane to 4 lane + 3 of the warp's 128
  int column;                // kind 1: the row this lane's row adds
};

__device__ __forceinline__ void fix_load(const TcFix& f, const TcGroup& g, int row0, int i0, FixState& q) {
  const int i = i0 + (threadIdx.x & 31);
  if (i < q.count) {
    q.token = __ldg(f.token + q.at + i);
    q.owner = (int)(__ldg(f.sorted + q.at + i) - (g.col0 + row0));
    q.lo = __ldg(f.lo + q.token);
  }
}

// Columns c to c + 31 of the warp's 128, which begin at column c0 of C.
__device__ __forceinline__ void fix_add_rows(const TcFix& f, const TcGroup& g, int row0, FixState& q, float* v, int c0,
                                             int c) {
  const int lane = threadIdx.x & 31;
  if (f.kind == 1) {
    if (q.column >= 0) {
      int k = 0;
      while (q.column >= f.first[k + 1]) ++k;
      fix_add(v, __ldg(f.lo + row0 + lane), static_cast<const __nv_bfloat16*>(f.w[k]) + (q.column - f.first[k]) * f.ld,
              c0 + c, f.ld);
    }
    __syncwarp();
    return;
  }
  for (int i0 = 0; i0 < q.count; i0 += 32) {  // in the order of the tokens
    if (q.count > 32) fix_load(f, g, row0, i0, q);
    for (int i = 0; i < 32 && i0 + i < q.count; ++i) {
      const int o = __shfl_sync(0xffffffffu, q.owner, i), t = __shfl_sync(0xffffffffu, q.token, i);
      const float w = __shfl_sync(0xffffffffu, q.lo, i);
      if (i0 + i < 2) {  // held in the warp's registers: 8 lanes have these 32 columns
        const uint2 h = i == 0 ? q.held[0] : q.held[1];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t a = __shfl_sync(0xffffffffu, h.x, c / 4 + k), b = __shfl_sync(0xffffffffu, h.y, c / 4 + k);
          if (lane == o) {
            v[4 * k] = fmaf(w, __uint_as_float(a << 16), v[4 * k]);
            v[4 * k + 1] = fmaf(w, __uint_as_float(a & 0xFFFF0000u), v[4 * k + 1]);
            v[4 * k + 2] = fmaf(w, __uint_as_float(b << 16), v[4 * k + 2]);
            v[4 * k + 3] = fmaf(w, __uint_as_float(b & 0xFFFF0000u), v[4 * k + 3]);
          }
        }
      } else if (lane == o) {
        fix_add(v, w, static_cast<const __nv_bfloat16*>(f.w[0]) + (long long)t * f.ld, c0 + c, f.ld);
      }
    }
    __syncwarp();
  }
}

template <bool F32>
struct EpiStore {
  using State = FixState;

  // Tiles that a join reads get kind 1 there.
  static __device__ __forceinline__ bool fixes(const TcArgs& p, const TcTile& x) {
    return p.fix.kind != 0 && !F32 && (x.slot < 0 || p.splits == 1);
  }

  static __device__ __forceinline__ State ahead(const TcArgs& p, const TcTile& x, int row0, int) {
    State q;
    q.at = q.count = 0;
    q.column = -1;
    const TcGroup& g = p.group[x.group];
    if (!fixes(p, x) || row0 >= g.M) return q;
    if (p.fix.kind == 1) {
      const int row = row0 + (threadIdx.x & 31);
      if (row < g.M) q.column = __ldg(p.fix.column + row);
    } else {
      const int* s = p.fix.start + g.part0 + row0 / 32;
      q.at = __ldg(s);
      q.count = __ldg(s + 1);  // less q.at, later
    }
    return q;
  }

  static __device__ __forceinline__ void more(const TcArgs& p, const TcTile& x, int row0, int half, State& q) {
    const TcFix& f = p.fix;
    const TcGroup& g = p.group[x.group];
    if (f.kind != 2 || !fixes(p, x) || row0 >= g.M) return;
    q.count -= q.at;
    if (q.count == 0) return;
    fix_load(f, g, row0, 0, q);
    const int c = x.n * 256 + half * 128 + 4 * (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = __shfl_sync(0xffffffffu, q.token, i);
      q.held[i] = make_uint2(0u, 0u);
      if (i < q.count && c + 4 <= f.ld)
        q.held[i] = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(f.w[0]) + (long long)t * f.ld + c));
    }
  }

  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row0, int half, uint32_t addr,
                                             uint8_t* buf, State& fix) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 256 + half * 128;
    const int rows = g.M - row0;
    const bool part = x.slot >= 0 && p.splits > 1;
    const bool on = fixes(p, x);
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
        if (on) fix_add_rows(p.fix, g, row0, fix, v, c0, c);
        tc_stage_bf16(buf, v, 0);
        tc_ld_ready(w);
        if (on) fix_add_rows(p.fix, g, row0, fix, w, c0, c + 32);
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

// Columns c to c + 7 of row r (lc and lr within the tile) as the products left them.
__device__ __forceinline__ void join_row(const JoinTiles& j, int tile, int r, int lr, int c, int lc, float4& a, float4& b) {
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
}

// A CTA takes 8 rows of a tile at a time, a thread 8 columns of one.
template <bool REST>
__device__ __forceinline__ void join_slab(const JoinTiles& j, int tile, int slab) {
  int m, n;
  tc_walk(tile, j.mt, j.nt, m, n);
  const bool vec = j.cols % 8 == 0 && ((uintptr_t)j.out & 15) == 0;
  const int lr = slab * 8 + (threadIdx.x >> 5), lc = (threadIdx.x & 31) * 8;
  const int r = m * 256 + lr, c = n * 256 + lc;
  if (r < j.rows && c < j.cols) {
    float4 a, b;
    join_row(j, tile, r, lr, c, lc, a, b);
    if (REST) {
      float4 x, y;
      join_row(j, tile, r + j.rest, lr + j.rest, c, lc, x, y);
      a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
      b = make_float4(b.x + y.x, b.y + y.y, b.z + y.z, b.w + y.w);
    }
    if (j.fix.kind) {
      const int col = __ldg(j.fix.column + r);
      if (col >= 0) {
        int k = 0;
        while (col >= j.fix.first[k + 1]) ++k;
        const float f = __ldg(j.fix.lo + r);
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(j.fix.w[k]) +
                                                             (col - j.fix.first[k]) * j.fix.ld + c));
        a.x = fmaf(f, __uint_as_float(u.x << 16), a.x);
        a.y = fmaf(f, __uint_as_float(u.x & 0xFFFF0000u), a.y);
        a.z = fmaf(f, __uint_as_float(u.y << 16), a.z);
        a.w = fmaf(f, __uint_as_float(u.y & 0xFFFF0000u), a.w);
        b.x = fmaf(f, __uint_as_float(u.z << 16), b.x);
        b.y = fmaf(f, __uint_as_float(u.z & 0xFFFF0000u), b.y);
        b.z = fmaf(f, __uint_as_float(u.w << 16), b.z);
        b.w = fmaf(f, __uint_as_float(u.w & 0xFFFF0000u), b.w);
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

template <bool REST>
__global__ void __launch_bounds__(kRowThreads)
    join_tiles_kernel(const __grid_constant__ JoinTiles j, int first, int slabs) {
  pdl_wait();
  pdl_next();
  for (int i = blockIdx.x; i < slabs; i += gridDim.x) join_slab<REST>(j, first + i / 32, i % 32);
}

cudaError_t launch_join_tiles(const JoinTiles& j, cudaStream_t s) {
  // without `acc` the whole tiles are in the output already
  const int first = j.acc ? 0 : j.full, tiles = j.mt * j.nt;
  if (first >= tiles || (!j.acc && j.splits == 1)) return cudaSuccess;
  const int slabs = (tiles - first) * 32;
  return launch_pdl(j.rest ? join_tiles_kernel<true> : join_tiles_kernel<false>, budget(slabs), kRowThreads, 0, s, j,
                    first, slabs);
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
