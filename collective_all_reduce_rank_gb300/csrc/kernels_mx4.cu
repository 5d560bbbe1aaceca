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
  int vec;
};

// A warp takes kMxTrips x 256 columns of a row at a time.
template <int DT>
__global__ void __launch_bounds__(kMxThreads) quantize_kernel(const QuantArgs a) {
  constexpr int ES = Elem<DT>::kSize;
  const int lane = threadIdx.x & 31;
  const size_t octets = (a.cols + 31) / 32 * 4, across = (a.cols + 127) / 128;
  const size_t pieces = (across * 16 + 32 * kMxTrips - 1) / (32 * kMxTrips);
  const size_t total = a.rows * pieces, step = (size_t)gridDim.x * (kMxThreads / 32);
  pdl_wait();
  for (size_t i = (size_t)blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const size_t row = i / pieces, o0 = (i - row * pieces) * (32 * kMxTrips) + lane;
    const char* src = a.x + row * a.cols * ES;
    float f[kMxTrips][8];
#pragma unroll
    for (int j = 0; j < kMxTrips; ++j) {
      const int v = octet_valid(o0 + 32 * j, a.cols);
      if (v > 0) {
        load8<DT>(src, o0 + 32 * j, v, a.vec, f[j]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[j][k] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < kMxTrips; ++j) mx_put8(f[j], a.codes, a.scales, row, o0 + 32 * j, octets, across, true);
  }
  pdl_next();
}

struct ReadArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  char* out;
  size_t rows, cols;
  int vec;
};

template <int DT>
__global__ void __launch_bounds__(kMxThreads) restore_kernel(const ReadArgs a) {
  constexpr int ES = Elem<DT>::kSize;
  const int lane = threadIdx.x & 31;
  const size_t octets = (a.cols + 31) / 32 * 4, across = (a.cols + 127) / 128, used = (a.cols + 7) / 8;
  const size_t pieces = (used + 32 * kMxTrips - 1) / (32 * kMxTrips);
  const size_t total = a.rows * pieces, step = (size_t)gridDim.x * (kMxThreads / 32);
  pdl_wait();
  for (size_t i = (size_t)blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const size_t row = i / pieces, o0 = (i - row * pieces) * (32 * kMxTrips) + lane;
    char* dst = a.out + row * a.cols * ES;
    uint32_t w[kMxTrips], b[kMxTrips];
#pragma unroll
    for (int j = 0; j < kMxTrips; ++j) {
      const size_t o = o0 + 32 * j;
      w[j] = o < used ? __ldg(reinterpret_cast<const uint32_t*>(a.codes + (row * octets + o) * 4)) : 0u;
      b[j] = o < used ? __ldg(a.scales + mx_scale_at(row, o / 4, across)) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kMxTrips; ++j) {
      const size_t o = o0 + 32 * j;
      if (o >= used) break;
      const float p = mx_power(b[j]);
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = mx_value2((w[j] >> (8 * k)) & 255u);
        f[2 * k] = v.x * p;
        f[2 * k + 1] = v.y * p;
      }
      store8<DT>(dst, o, octet_valid(o, a.cols), a.vec, f);
    }
  }
  pdl_next();
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
  int vec;
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

// 1 / sqrt(sum / count + eps): the special function's value, improved by one
// Newton step whose residual 1 - x r^2 is taken from the pairs.
__device__ __forceinline__ float pair_rstd(Pair sum, float count, float eps) {
  const float q = __fdiv_rn(sum.hi, count);
  const float rest = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, count, sum.hi), sum.lo), count);
  Pair x = pair_add({q, rest}, {eps, 0.f});
  const float r = rsqrtf(x.hi);
  if (!(r > 0.f) || r > 3e38f) return r;  // 0, infinite or NaN already
  const float t = __fmul_rn(r, r), tl = __fmaf_rn(r, r, -t);
  const float p = __fmul_rn(x.hi, t);
  const float pl = __fadd_rn(__fmaf_rn(x.hi, t, -p), __fmaf_rn(x.lo, t, __fmul_rn(x.hi, tl)));
  const float e = __fsub_rn(__fsub_rn(1.f, p), pl);
  return __fmaf_rn(__fmul_rn(0.5f, r), e, r);
}

// One CTA per row (or every gridDim-th row).  U octets a thread in registers;
// U == 0: long rows, kept in shared memory.
template <int DT, int U>
__global__ void __launch_bounds__(1024) norm_mx4_kernel(const __grid_constant__ NormMxArgs a) {
  constexpr int ES = Elem<DT>::kSize, PU = Elem<DT>::kPerUnit;
  extern __shared__ float srow[];
  __shared__ Pair part[2][32];
  const size_t hidden = a.hidden, octets = (hidden + 31) / 32 * 4, across = (hidden + 127) / 128;
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
  const int trips = U ? U : (int)((across * 16 + threads - 1) / threads);
  int flip = 0;
  pdl_wait();
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const size_t off = row * hidden * ES;
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
            if (k < a.n) x[k] = load_row<DT>(static_cast<const char*>(a.in[k]) + off, u, vh, a.vec);
          if (a.residual) r = load_row<DT>(a.residual + off, u, vh, a.vec);
          Acc acc;
          acc_init<DT>(acc, x[0]);
#pragma unroll
          for (int k = 1; k < kMaxRanks; ++k)
            if (k < a.n) acc_add<DT>(acc, x[k]);
          if (a.residual) acc_add<DT>(acc, r);
#pragma unroll
          for (int i = 0; i < PU; ++i) s[h * PU + i] = __uint_as_float(acc.w[i]);
        }
        if (a.residual_out) store8<DT>(a.residual_out + off, o, v, a.vec, s);
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
    Pair tot = (tid & 31) < warps ? part[flip][tid & 31] : Pair{0.f, 0.f};
    tot = pair_reduce(tot);
    const float inv = pair_rstd(tot, (float)hidden, a.eps);
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
        if (DT == RRA_BFLOAT16 && a.vec) {
          unit_floats<DT>(__ldg(static_cast<const uint4*>(a.gamma) + o), g);
        } else {
          load8<DT>(static_cast<const char*>(a.gamma), o, v, a.vec, g);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = i < v ? __fmul_rn(__fmul_rn(s[i], inv), g[i]) : 0.f;
      }
      mx_put8(s, a.codes, a.scales, row, o, octets, across, true);
    }
  }
  pdl_next();
}

template <int DT>
cudaError_t norm_dt(const NormMxArgs& a, cudaStream_t s) {
  // one octet a thread while that fits a CTA and the rows are few (one row's
  // latency is then the call's), two for many rows or longer ones
  const size_t lanes = (a.hidden + 127) / 128 * 16;  // octets up to the last tile's end
  const int grid = budget(a.rows);
  const auto threads = [&](int u) { return (int)(((lanes + u - 1) / u + 31) / 32 * 32); };
  if (lanes <= 1024 && (a.rows <= 2 * (size_t)device_sms() || lanes <= 256))
    return launch_pdl(norm_mx4_kernel<DT, 1>, grid, threads(1), 0, s, a);
  if (lanes <= 2048) return launch_pdl(norm_mx4_kernel<DT, 2>, grid, threads(2), 0, s, a);
  constexpr auto kern = norm_mx4_kernel<DT, 0>;
  const cudaError_t e = raise_smem<kern>(200 * 1024 + 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, 512, (a.hidden + 31) / 32 * 32 * sizeof(float), s, a);
}

// CTAs that fill the GPU a few times over, or fewer.
int stream_grid(size_t pieces) {
  const size_t ctas = (pieces + kMxThreads / 32 - 1) / (kMxThreads / 32);
  const size_t most = (size_t)device_sms() * 16;
  return budget(ctas < most ? ctas : most);
}

}  // namespace

cudaError_t launch_mx4_quantize(int dt, bool vec, const void* x, void* codes, void* scales, size_t rows, size_t cols,
                                cudaStream_t s) {
  const QuantArgs a{static_cast<const char*>(x), static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), rows,
                    cols, vec};
  const int grid = stream_grid(rows * (((cols + 127) / 128 * 16 + 32 * kMxTrips - 1) / (32 * kMxTrips)));
  return dt == RRA_BFLOAT16 ? launch_pdl(quantize_kernel<RRA_BFLOAT16>, grid, kMxThreads, 0, s, a)
                            : launch_pdl(quantize_kernel<RRA_FLOAT32>, grid, kMxThreads, 0, s, a);
}

cudaError_t launch_mx4_restore(int dt, bool vec, const void* codes, const void* scales, void* out, size_t rows,
                               size_t cols, cudaStream_t s) {
  const ReadArgs a{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), static_cast<char*>(out),
                   rows, cols, vec};
  const int grid = stream_grid(rows * (((cols + 7) / 8 + 32 * kMxTrips - 1) / (32 * kMxTrips)));
  return dt == RRA_BFLOAT16 ? launch_pdl(restore_kernel<RRA_BFLOAT16>, grid, kMxThreads, 0, s, a)
                            : launch_pdl(restore_kernel<RRA_FLOAT32>, grid, kMxThreads, 0, s, a);
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
  a.vec = vec;
  return dt == RRA_BFLOAT16 ? norm_dt<RRA_BFLOAT16>(a, s) : norm_dt<RRA_FLOAT32>(a, s);
}

}  // namespace rra
