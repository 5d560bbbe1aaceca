// kernels_mx4.cu -- matrices in MX4 (mx4.cuh): quantised, read back, and made
// by the fused all-reduce + residual + RMSNorm.
//
//   s = sum_k x_k (float32, ascending ranks) + residual, residual' = s,
//   q = 1 / sqrt(mean s^2 + eps), y = (s q) gamma -> MX4
//
// A 4-bit code turns a last-bit difference at one of its borders into a whole
// step, so y is fixed to the bit: s is added in rank order, q is the float32
// nearest to its exact value (the squares are summed as pairs of float32, error
// below 2^-40) and both products round to float32.
//
// All three are bound by HBM on large matrices: one pass, loads of several
// octets in flight a lane.  16384 x 5120 bf16 quantised in 39 us and read back
// in 32 (5.5 and 6.6 TB/s), the sum of 8 ranks' 4096 x 5120 with a residual 72
// us, of float32 143 (6.0 TB/s both).  Small ones are latency: 8 x 5120 x 8 ranks 3.6 us, 1283 x
// 1027 float32, whose rows start on no 16 bytes, 4.6 and 4.5.
#include "mx4.cuh"
#include "pdl.cuh"
#include "serve_host.h"
#include "smem_limit.h"

namespace rra {

namespace {

constexpr int kMxThreads = 256;
constexpr int kMxTrips = 4;  // octets of a lane whose loads are in flight together

struct QuantArgs {
  const char* x;
  uint8_t* codes;
  uint8_t* scales;
  size_t rows, cols;
};

// Piece i of rows cut into `pieces`: 32-bit division where it will do (64-bit
// division is some 100 instructions, as many as an octet's whole work).
__device__ __forceinline__ size_t piece_row(size_t i, uint32_t pieces) {
  if (pieces == 1) return i;
  return (i >> 32) == 0 ? (uint32_t)i / pieces : i / pieces;
}

// A warp takes kMxTrips x 256 columns of a row at a time.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kMxThreads) quantize_kernel(const QuantArgs a) {
  constexpr int ES = Elem<DT>::kSize;
  const int lane = threadIdx.x & 31;
  const uint32_t pieces = (uint32_t)(((a.cols + 127) / 128 * 16 + 32 * kMxTrips - 1) / (32 * kMxTrips));
  const size_t total = a.rows * pieces, step = (size_t)gridDim.x * (kMxThreads / 32);
  pdl_wait();
  for (size_t i = (size_t)blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const size_t row = piece_row(i, pieces);
    const uint32_t o0 = (uint32_t)(i - row * pieces) * (32 * kMxTrips) + lane;
    const char* src = a.x + row * a.cols * ES;
    const MxRow r = mx_from(mx_row(a.codes, a.scales, row, a.cols), o0);
    if constexpr (DT == RRA_BFLOAT16 && VEC) {
      const uint32_t units = (uint32_t)(a.cols / 8);
      uint4 x[kMxTrips];
#pragma unroll
      for (int j = 0; j < kMxTrips; ++j)
        x[j] = o0 + 32 * j < units ? ld_stream(src + (size_t)(o0 + 32 * j) * 16) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j = 0; j < kMxTrips; ++j) {
        if (o0 - lane + 32 * j >= r.ends) break;
        mx_put8(x[j], r, o0 + 32 * j);
      }
    } else {
      float f[kMxTrips][8];
#pragma unroll
      for (int j = 0; j < kMxTrips; ++j) {
        const int v = octet_valid(o0 + 32 * j, a.cols);
        if (v > 0) {
          load8<DT>(src, o0 + 32 * j, v, VEC, f[j]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[j][k] = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < kMxTrips; ++j) {
        if (o0 - lane + 32 * j >= r.ends) break;
        mx_put8(f[j], r, o0 + 32 * j);
      }
    }
  }
  pdl_next();
}

struct ReadArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  char* out;
  size_t rows, cols;
};

// VEC: rows of whole aligned 16-byte units, an octet of columns a lane.  Others:
// a lane stores every 32nd column of 256, so that a warp's stores stay together,
// and finds its codes in the words that the lanes hold (1283 x 1027 float32 6.8
// us with an octet a lane).
template <int DT, bool VEC>
__global__ void __launch_bounds__(kMxThreads) restore_kernel(const ReadArgs a) {
  constexpr int ES = Elem<DT>::kSize;
  const int lane = threadIdx.x & 31;
  const uint32_t used = (uint32_t)((a.cols + 7) / 8), pieces = (used + 32 * kMxTrips - 1) / (32 * kMxTrips);
  const size_t total = a.rows * pieces, step = (size_t)gridDim.x * (kMxThreads / 32);
  pdl_wait();
  for (size_t i = (size_t)blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const size_t row = piece_row(i, pieces);
    const uint32_t o0 = (uint32_t)(i - row * pieces) * (32 * kMxTrips) + lane;
    char* dst = a.out + row * a.cols * ES;
    const MxRow r = mx_from(mx_row(a.codes, a.scales, row, a.cols), o0);
    uint32_t w[kMxTrips], b[kMxTrips];
#pragma unroll
    for (int j = 0; j < kMxTrips; ++j) {
      const uint32_t o = o0 + 32 * j;
      w[j] = o < used ? __ldg(r.codes + o) : 0u;
      b[j] = o < used ? __ldg(r.scales + (o / 16) * 512 + (o / 4) % 4) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kMxTrips; ++j) {
      const uint32_t o = o0 + 32 * j;
      if (VEC) {
        if (o >= used) break;
        float f[8];
        mx_value8(w[j], mx_power(b[j]), f);
        store8<DT>(dst, o, octet_valid(o, a.cols), true, f);
      } else {
        if (o - lane >= used) break;
#pragma unroll
        for (int q = 0; q < 8; ++q) {  // column 32 q + lane of the 256
          const uint32_t word = __shfl_sync(0xffffffffu, w[j], 4 * q + (lane >> 3));
          const uint32_t byte = __shfl_sync(0xffffffffu, b[j], 4 * q);
          const float v = mx_value(word >> (4 * (lane & 7))) * mx_power(byte);
          const size_t col = (size_t)(o - lane) * 8 + 32 * q + lane;
          if (col < a.cols) {
            if (DT == RRA_BFLOAT16)
              reinterpret_cast<__nv_bfloat16*>(dst)[col] = __float2bfloat16_rn(v);
            else
              reinterpret_cast<float*>(dst)[col] = v;
          }
        }
      }
    }
  }
  pdl_next();
}

template <int DT>
cudaError_t quantize_go(const QuantArgs& a, bool vec, int grid, cudaStream_t s) {
  return vec ? launch_pdl(quantize_kernel<DT, true>, grid, kMxThreads, 0, s, a)
             : launch_pdl(quantize_kernel<DT, false>, grid, kMxThreads, 0, s, a);
}

template <int DT>
cudaError_t restore_go(const ReadArgs& a, bool vec, int grid, cudaStream_t s) {
  return vec ? launch_pdl(restore_kernel<DT, true>, grid, kMxThreads, 0, s, a)
             : launch_pdl(restore_kernel<DT, false>, grid, kMxThreads, 0, s, a);
}

// ---------------------------------------------------------------------------
// all-reduce + residual + RMSNorm
// ---------------------------------------------------------------------------

struct NormMxArgs {
  const void* in[kMaxRanks];
  const void* gamma;
  const char* residual;  // null: none
  char* residual_out;
  uint8_t* codes;
  uint8_t* scales;
  size_t rows, hidden;
  float eps;
  int n;
};

// A sum held as an unevaluated pair of float32.
struct Pair {
  float hi, lo;
};

__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const float t = __fadd_rn(a.hi, b.hi), z = __fsub_rn(t, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(t, z)), __fsub_rn(b.hi, z));
  return {t, __fadd_rn(__fadd_rn(a.lo, b.lo), e)};
}

__device__ __forceinline__ Pair pair_square(Pair a, float s) {
  const float p = __fmul_rn(s, s);
  return pair_add(a, {p, __fmaf_rn(s, s, -p)});
}

__device__ __forceinline__ Pair pair_reduce(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Pair w{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
    // the lower lane's first: every lane gets the same bits
    v = threadIdx.x & o ? pair_add(w, v) : pair_add(v, w);
  }
  return v;
}

// 1 / sqrt(sum / count + eps): the special function's value r, improved by one
// Newton step whose residual 1 - x r^2 is taken from the pairs, as 1 - (x r) r:
// r^2 may be out of float32's range, x r is not.
__device__ __forceinline__ float pair_rstd(Pair sum, float count, float eps) {
  const float q = __fdiv_rn(sum.hi, count);
  const float rest = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, count, sum.hi), sum.lo), count);
  Pair x = pair_add({q, rest}, {eps, 0.f});
  const float r = rsqrtf(x.hi);
  if (!(r > 0.f) || r > 3e38f) return r;  // 0, infinite or NaN already
  const float h = __fmul_rn(x.hi, r), hl = __fmaf_rn(x.lo, r, __fmaf_rn(x.hi, r, -h));
  const float p = __fmul_rn(h, r), pl = __fmaf_rn(hl, r, __fmaf_rn(h, r, -p));
  const float e = __fsub_rn(__fsub_rn(1.f, p), pl);
  return __fmaf_rn(__fmul_rn(0.5f, r), e, r);
}

// The same of a sum and an eps below 2^-60, whose quotient by count may be below
// float32's normal numbers: both are taken times 2^100.  A call of its own: in
// line it made rows of two octets a thread spill (4096 x 5120 x 8 ranks float32
// 141 -> 149 us).
__device__ __noinline__ float pair_rstd_small(Pair sum, float count, float eps) {
  constexpr float kUp = 0x1p100f;
  return __fmul_rn(0x1p50f, pair_rstd({__fmul_rn(sum.hi, kUp), __fmul_rn(sum.lo, kUp)}, count, __fmul_rn(eps, kUp)));
}

// acc_add with the bfloat16 widened by the addition itself.
template <int DT>
__device__ __forceinline__ void add_unit(Acc& a, const uint4& v) {
  if constexpr (DT == RRA_BFLOAT16) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\nadd.rn.f32.bf16 %0, l, %0;\nadd.rn.f32.bf16 %1, h, %1;\n}"
          : "+r"(a.w[2 * i]), "+r"(a.w[2 * i + 1])
          : "r"(x[i]));
  } else {
    acc_add<DT>(a, v);
  }
}

// One CTA per row (or every gridDim-th row).  U octets a thread in registers;
// U == 0: long rows, kept in shared memory.  (U == 2 has 64 registers a thread for
// two CTAs of 512 an SM: rows that start on no 16 bytes spill 80 to 108 bytes.)
template <int DT, int U, bool VEC>
__global__ void __launch_bounds__(U == 1 ? 1024 : 512, U == 2 ? 2 : 1) norm_mx4_kernel(const __grid_constant__ NormMxArgs a) {
  constexpr int ES = Elem<DT>::kSize, PU = Elem<DT>::kPerUnit;
  extern __shared__ float srow[];
  __shared__ Pair part[2][32];
  __shared__ float rstd[2];
  const size_t hidden = a.hidden, octets = (hidden + 31) / 32 * 4, across = (hidden + 127) / 128;
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
  const int trips = U ? U : (int)((across * 16 + threads - 1) / threads);
  int flip = 0;
  pdl_wait();
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const size_t off = row * hidden * ES;
    const MxRow out = mx_row(a.codes, a.scales, row, hidden);
    float f[U ? U : 1][8];
    Pair ss{0.f, 0.f};
#pragma unroll
    for (int j = 0; j < trips; ++j) {
      float* s = f[U ? j : 0];
      const size_t o = (size_t)j * threads + tid;
      const int v = octet_valid(o, hidden);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 0.f;
      if (v > 0) {
        // a 16-byte unit of every rank in flight before its first addition
#pragma unroll
        for (int h = 0; h < 8 / PU; ++h) {
          const int vh = min(v - h * PU, PU);
          if (vh <= 0) break;
          const size_t u = o * (8 / PU) + h;
          uint4 x[kMaxRanks], r = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int k = 0; k < kMaxRanks; ++k)
            if (k < a.n) x[k] = load_row<DT>(static_cast<const char*>(a.in[k]) + off, u, vh, VEC);
          if (a.residual) r = load_row<DT>(a.residual + off, u, vh, VEC);
          Acc acc;
          acc_init<DT>(acc, x[0]);
#pragma unroll
          for (int k = 1; k < kMaxRanks; ++k)
            if (k < a.n) add_unit<DT>(acc, x[k]);
          if (a.residual) add_unit<DT>(acc, r);
#pragma unroll
          for (int i = 0; i < PU; ++i) s[h * PU + i] = __uint_as_float(acc.w[i]);
        }
        if (a.residual_out) store8<DT>(a.residual_out + off, o, v, VEC, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = pair_square(ss, i < v ? s[i] : 0.f);
      }
      if (U == 0 && o < octets) {
#pragma unroll
        for (int i = 0; i < 8; ++i) srow[o * 8 + i] = s[i];
      }
    }
    ss = pair_reduce(ss);
    if ((tid & 31) == 0) part[flip][tid >> 5] = ss;
    __syncthreads();
    if (tid < 32) {  // one warp for all: the others' issue slots go to other rows
      const Pair sum = pair_reduce(tid < warps ? part[flip][tid] : Pair{0.f, 0.f});
      const float count = (float)hidden;
      const float q = fmaxf(sum.hi, a.eps) < 0x1p-60f ? pair_rstd_small(sum, count, a.eps) : pair_rstd(sum, count, a.eps);
      if (tid == 0) rstd[flip] = q;
    }
    __syncthreads();
    const float inv = rstd[flip];
#pragma unroll
    for (int j = 0; j < trips; ++j) {
      float* s = f[U ? j : 0];
      const size_t o = (size_t)j * threads + tid;
      const int v = octet_valid(o, hidden);
      if (U == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = o < octets ? srow[o * 8 + i] : 0.f;
      }
      if (v > 0) {
        float g[8];
        if (DT == RRA_BFLOAT16 && VEC) {
          unit_floats<DT>(__ldg(static_cast<const uint4*>(a.gamma) + o), g);
        } else {
          load8<DT>(static_cast<const char*>(a.gamma), o, v, VEC, g);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = i < v ? __fmul_rn(__fmul_rn(s[i], inv), g[i]) : 0.f;
      }
      mx_put8(s, out, (uint32_t)o);
    }
  }
  pdl_next();
}

template <int DT, bool VEC>
cudaError_t norm_dt(const NormMxArgs& a, cudaStream_t s) {
  // one octet a thread while that fits a CTA and the rows are few (one row's
  // latency is then the call's), two for many rows, four for longer ones
  const size_t lanes = (a.hidden + 127) / 128 * 16;  // octets up to the last tile's end
  const int grid = budget(a.rows);
  const auto threads = [&](int u) { return (int)(((lanes + u - 1) / u + 31) / 32 * 32); };
  if (lanes <= 1024 && (a.rows <= 2 * (size_t)device_sms() || lanes <= 256))
    return launch_pdl(norm_mx4_kernel<DT, 1, VEC>, grid, threads(1), 0, s, a);
  if (lanes <= 1024) return launch_pdl(norm_mx4_kernel<DT, 2, VEC>, grid, threads(2), 0, s, a);
  if (lanes <= 2048) return launch_pdl(norm_mx4_kernel<DT, 4, VEC>, grid, threads(4), 0, s, a);
  constexpr auto kern = norm_mx4_kernel<DT, 0, VEC>;
  const cudaError_t e = raise_smem<kern>(200 * 1024 + 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, 512, (a.hidden + 31) / 32 * 32 * sizeof(float), s, a);
}

// CTAs that fill the GPU a few times over, or fewer.
int stream_grid(size_t pieces) {
  const size_t ctas = (pieces + kMxThreads / 32 - 1) / (kMxThreads / 32);
  const size_t most = (size_t)device_sms() * 64;
  return budget(ctas < most ? ctas : most);
}

}  // namespace

cudaError_t launch_mx4_quantize(int dt, bool vec, const void* x, void* codes, void* scales, size_t rows, size_t cols,
                                cudaStream_t s) {
  const QuantArgs a{static_cast<const char*>(x), static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), rows,
                    cols};
  const int grid = stream_grid(rows * (((cols + 127) / 128 * 16 + 32 * kMxTrips - 1) / (32 * kMxTrips)));
  return dt == RRA_BFLOAT16 ? quantize_go<RRA_BFLOAT16>(a, vec, grid, s) : quantize_go<RRA_FLOAT32>(a, vec, grid, s);
}

cudaError_t launch_mx4_restore(int dt, bool vec, const void* codes, const void* scales, void* out, size_t rows,
                               size_t cols, cudaStream_t s) {
  const ReadArgs a{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), static_cast<char*>(out),
                   rows, cols};
  const int grid = stream_grid(rows * (((cols + 7) / 8 + 32 * kMxTrips - 1) / (32 * kMxTrips)));
  return dt == RRA_BFLOAT16 ? restore_go<RRA_BFLOAT16>(a, vec, grid, s) : restore_go<RRA_FLOAT32>(a, vec, grid, s);
}

cudaError_t launch_norm_mx4(int n, int dt, bool vec, const void* const* in, const void* residual, void* residual_out,
                            const void* gamma, size_t rows, size_t hidden, float eps, void* codes, void* scales,
                            cudaStream_t s) {
  NormMxArgs a{};
  for (int r = 0; r < n; ++r) a.in[r] = in[r];
  a.gamma = gamma;
  a.residual = static_cast<const char*>(residual);
  a.residual_out = static_cast<char*>(residual_out);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  a.rows = rows;
  a.hidden = hidden;
  a.eps = eps;
  a.n = n;
  if (dt == RRA_BFLOAT16) return vec ? norm_dt<RRA_BFLOAT16, true>(a, s) : norm_dt<RRA_BFLOAT16, false>(a, s);
  return vec ? norm_dt<RRA_FLOAT32, true>(a, s) : norm_dt<RRA_FLOAT32, false>(a, s);
}

}  // namespace rra
