// kernels_mx4_few.cu -- products of MX4 matrices for few tokens (up to 128,
// mx4_few_most below), where reading the weights is the time.
//
// The weights are the product's long side: a CTA takes 128 weight rows (gated:
// 128 of the gate's and the same 128 of the up projection's) against all tokens
// as its 16 to 128 columns, so that a tensor-memory lane is a weight row and
// every byte of the weights is staged once.  A ring of 256-column stages keeps
// up to 200 KB a SM on its way.
//
// Few weight rows (a row-parallel layer's 5120 are 40 tiles) leave SMs without
// a tile, so a cluster of up to 8 CTAs shares a tile's K axis: each sends its
// float32 sums through distributed shared memory to the CTA that owns the
// column, which adds them in the order of K.  Nothing depends on timing.
//
// A gated block's 32 columns are a warp's 32 lanes.  Of up to four tokens the
// largest value is one warp reduction, the codes four words of lanes or-ed
// together; of more, lanes exchange rows for tokens.
//
// Bound by HBM: 1 token x 131072 x 5120 58 us (6.1 TB/s), x 5120 x 13824 row-
// parallel 11 us, gated 16 (3.3 and 4.8 TB/s: 108 tiles for 152 SMs, and a
// kernel's 3 us of start and end).
//
// Roles (8 warps): warp 0 loads, warp 1 issues, warp 2 owns the tensor memory,
// warps 4-7 are the epilogue.
#include "act.cuh"
#include "mx4_mma.cuh"

namespace rra {

namespace {

constexpr int kFewThreads = 256;
constexpr int kEpiWarps = 4;
constexpr int kRows = 128;
constexpr int kWCodes = kRows * 128, kWScales = 1024, kXScales = 1024;
constexpr int kMost = 224 * 1024;  // dynamic shared memory: ring, sums of a cluster, alignment
constexpr int kMaxSplit = 8;

template <int N, bool GATED>
struct Few {
  static constexpr int G = GATED ? 2 : 1;
  static constexpr int kStage = G * (kWCodes + kWScales) + N * 128 + kXScales;
  static constexpr int kBufs = 2 * G * N <= 480 ? 2 : 1;
  static constexpr int kColX = 512 - 8, kColW = kColX - 8 * G;
  static_assert(kBufs * G * N <= kColW, "accumulators and scales fit tensor memory");
  // every CTA's share of the owned columns
  static int sums(int split) { return split > 1 ? split * ((N + split - 1) / split) * G * kRows * 4 : 0; }
  static int stages(int split) {
    const int n = (kMost - 1024 - sums(split)) / kStage;
    return n < kTcMaxStages ? n : kTcMaxStages;
  }
};

struct FewShared : TcShared {
  alignas(8) uint64_t sums_full;
  alignas(8) uint64_t sums_empty;
};

__device__ __forceinline__ void few_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Arrive at a barrier of CTA `cta` of the cluster, publishing this warp's
// stores to that CTA's shared memory.
__device__ __forceinline__ void few_arrive(uint32_t bar, uint32_t cta) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(tc_mapa(bar, cta)) : "memory");
}

__device__ __forceinline__ void few_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// 32 lanes x 16 columns
__device__ __forceinline__ void few_ld16(uint32_t addr, float* v) {
  uint32_t r[16];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ int few_group(const Mx4Args& p, int t) {
  int g = 0;
  while (g + 1 < p.ngroups && t >= p.group[g + 1].tile0) ++g;
  return g;
}

// One token's value of this lane's weight row (gated: of its gate and up
// rows): stored, or quantised with the other 31 lanes' and stored.  The whole
// warp calls this.
template <int ACT>
__device__ __forceinline__ void few_put(const Mx4Args& p, const Mx4Group& g, int row0, int token, float a, float b) {
  const int lane = threadIdx.x & 31, row = row0 + lane;
  if constexpr (ACT < 0) {
    if (row >= g.rows) return;
    const long long at = (long long)token * g.ld + row;
    if (p.f32)
      static_cast<float*>(g.out)[at] = a;
    else
      static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16_rn(a);
  } else {
    float unused;
    const float v = row < g.rows ? a * gate_sigma<ACT>(a, &unused) * b : 0.f;
    const uint32_t byte = mx_scale(__reduce_max_sync(0xffffffffu, mx_abs(v)));
    uint32_t w = byte == kMxNan ? 0u : mx_code(v * mx_inverse(byte)) << (4 * (lane & 7));
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    if ((lane & 7) == 0 && row0 < g.rows)
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(g.out) + (long long)token * g.ld + row0 / 2 + lane / 2) = w;
    if (lane == 0) g.out_scales[mx_scale_at((size_t)token, (size_t)(row0 / 32), (size_t)g.across)] = (uint8_t)byte;
  }
}

// n of 16 tokens from `token` on, side by side.  Gated: rows and tokens change
// places between lanes, so that a lane has half a token's block (a reduction, a
// conversion and three exchanges a token: 16 tokens 2.2 us, this way 0.9).
template <int ACT>
__device__ __forceinline__ void few_put16(const Mx4Args& p, const Mx4Group& g, int row0, int token, int n,
                                          const float* a, const float* b) {
  const int lane = threadIdx.x & 31, row = row0 + lane;
  if constexpr (ACT < 0) {
    const bool live = row < g.rows;
    const long long at = (long long)token * g.ld + row;
    if (p.f32) {
      float* o = static_cast<float*>(g.out) + at;
#pragma unroll
      for (int j = 0; j < 16; ++j, o += g.ld)
        if (live && j < n) *o = a[j];
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g.out) + at;
#pragma unroll
      for (int j = 0; j < 16; ++j, o += g.ld)
        if (live && j < n) *o = __float2bfloat16_rn(a[j]);
    }
  } else {
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float unused;
      v[j] = row < g.rows ? a[j] * gate_sigma<ACT>(a[j], &unused) * b[j] : 0.f;
    }
    // 16 x 16 values change places: lane l has rows 16 (l / 16) + j of token l % 16
#pragma unroll
    for (int m = 8; m > 0; m /= 2)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (j & m) continue;
        const bool up = lane & m;
        const float got = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + m], m);
        v[j] = up ? got : v[j];
        v[j + m] = up ? v[j + m] : got;
      }
    uint32_t most = max(mx_amax8(v), mx_amax8(v + 8));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 16));
    const uint32_t byte = mx_scale(most);
    const float inv = mx_inverse(byte);
    const uint2 w = make_uint2(mx_code8(v, inv, byte == kMxNan), mx_code8(v + 8, inv, byte == kMxNan));
    const int t = lane & 15;
    if (t < n && row0 < g.rows)
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(g.out) + (long long)(token + t) * g.ld + row0 / 2 + lane / 16 * 8) = w;
    if (lane < n) g.out_scales[mx_scale_at((size_t)(token + t), (size_t)(row0 / 32), (size_t)g.across)] = (uint8_t)byte;
  }
}

template <int N, int ACT>
__global__ void __launch_bounds__(kFewThreads, 1) mx4_few_kernel(const __grid_constant__ Mx4Args p) {
  using F = Few<N, (ACT >= 0)>;
  constexpr int G = F::G;
  extern __shared__ uint8_t raw[];
  __shared__ FewShared sh;
  const uint32_t ring = (tc_smem(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split, nstages = p.stages;
  const uint32_t rank = S > 1 ? tc_cta_rank() : 0;
  const int cluster = blockIdx.x / S, clusters = gridDim.x / S;
  const int k0 = (int)((long long)p.kblocks * rank / S), k1 = (int)((long long)p.kblocks * (rank + 1) / S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < nstages; ++s) {
      tc_bar_init(tc_smem(&sh.full[s]), 1);
      tc_bar_init(tc_smem(&sh.empty[s]), 1);
    }
    for (int b = 0; b < F::kBufs; ++b) {
      tc_bar_init(tc_smem(&sh.acc_full[b]), 1);
      tc_bar_init(tc_smem(&sh.acc_empty[b]), kEpiWarps);
    }
    tc_bar_init(tc_smem(&sh.sums_full), kEpiWarps * S);
    tc_bar_init(tc_smem(&sh.sums_empty), kEpiWarps * S);
    sh.give_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(&sh.tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  pdl_next();

  // a stage: codes of W (twice if gated), of X, scales of W, of X
  constexpr uint32_t kX = G * kWCodes, kSW = kX + N * 128, kSX = kSW + G * kWScales;
  uint32_t issued = 0;
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = tc_smem(&sh.full[0]), empty0 = tc_smem(&sh.empty[0]);
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
      for (int t = cluster; t < p.tiles && ok; t += clusters) {
        const int g = few_group(p, t);
        const int tile = t - p.group[g].tile0;
        int seg = 0;
        for (int k = k0; k < k1; ++k, ++issued) {
          while (seg + 1 < p.nsegs && k >= p.seg_k0[seg + 1]) ++seg;
          const int kk = k - p.seg_k0[seg];
          const int w = p.nsegs > 1 ? seg : p.group[g].w;
          if (!tc_wait(empty0 + 8 * s, parity, &sh, p.status, 1)) {
            ok = false;
            break;
          }
          const uint32_t at = ring + s * F::kStage, bar = full0 + 8 * s;
          tc_bar_expect(bar, F::kStage);
#pragma unroll
          for (int i = 0; i < G; ++i) {
            mx4_load(&p.w[w + i], at + i * kWCodes, bar, kk * 128, tile * kRows);
            mx4_load(&p.ws[w + i], at + kSW + i * kWScales, bar, kk * 256, tile);
          }
          mx4_load(&p.x[seg], at + kX, bar, kk * 128, 0);
          mx4_load(&p.xs[seg], at + kSX, bar, kk * 256, 0);
          if (++s == nstages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
      for (int i = 0; i < nstages && ok; ++i) {  // the last releases land before this CTA leaves
        ok = tc_wait(empty0 + 8 * s, parity, &sh, p.status, 5);
        if (++s == nstages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // the whole warp walks the stages, one lane issues (kernels_mx4_product.cu)
    const bool lead = mx4_elect();
    uint32_t tile = 0, round = 0;
    int s = 0;
    bool ok = true;
    for (int t = cluster; t < p.tiles && ok; t += clusters, ++tile) {
      const uint32_t b = tile % F::kBufs, d = tmem + b * G * N;
      ok = __all_sync(0xffffffffu, tc_wait(tc_smem(&sh.acc_empty[b]), ((tile / F::kBufs) & 1) ^ 1, &sh, p.status, 2));
      if (!ok) break;
      tc_fence_after();
      for (int k = k0; k < k1; ++k) {
        ok = __all_sync(0xffffffffu, tc_wait(tc_smem(&sh.full[s]), round & 1, &sh, p.status, 3));
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = ring + s * F::kStage;
        if (lead) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < G; ++i)
              mx4_put_scales(tmem + F::kColW + 8 * i + 4 * j, at + kSW + i * kWScales + 512 * j);
            mx4_put_scales(tmem + F::kColX + 4 * j, at + kSX + 512 * j);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g)
              mx4_mma<false>(d + g * N, tc_desc<false>(at + g * kWCodes + 32 * i), tc_desc<false>(at + kX + 32 * i),
                             mx4_idesc(kRows, N) | mx4_idesc_scales(2 * (i & 1)), tmem + F::kColW + 8 * g + 4 * (i >> 1),
                             tmem + F::kColX + 4 * (i >> 1), (uint32_t)(k > k0 || i > 0));
          few_commit(tc_smem(&sh.empty[s]));
        }
        __syncwarp();
        if (++s == nstages) {
          s = 0;
          ++round;
        }
      }
      if (ok && lead) few_commit(tc_smem(&sh.acc_full[b]));
      __syncwarp();
    }
  } else if (warp >= 4) {
    const int quad = warp & 3, lanes = quad * 32;
    const int share = (N + S - 1) / S;  // columns a CTA of the cluster owns
    const uint32_t sums = ring + nstages * F::kStage;  // [CTA of the K axis][gate, up][owned column][row]
    const float* mine = reinterpret_cast<const float*>(raw + (sums - tc_smem(raw)));
    uint32_t tile = 0;
    for (int t = cluster; t < p.tiles; t += clusters, ++tile) {
      const uint32_t b = tile % F::kBufs;
      if (!__all_sync(0xffffffffu, tc_wait(tc_smem(&sh.acc_full[b]), (tile / F::kBufs) & 1, &sh, p.status, 4))) break;
      tc_fence_after();
      const Mx4Group& g = p.group[few_group(p, t)];
      const int row0 = (t - g.tile0) * kRows + lanes;
      const uint32_t addr = tmem + b * G * N + ((uint32_t)lanes << 16);
      if (S == 1) {
#pragma unroll 1
        for (int c = 0; c < N; c += 16) {
          if (c >= p.tokens) break;
          float v[G][16];
#pragma unroll
          for (int i = 0; i < G; ++i) few_ld16(addr + i * N + c, v[i]);
          const int n = min(p.tokens - c, 16);
          if (n <= 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < n) few_put<ACT>(p, g, row0, c + j, v[0][j], v[G - 1][j]);
          } else {
            few_put16<ACT>(p, g, row0, c, n, v[0], v[G - 1]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tc_bar_arrive_remote(tc_smem(&sh.acc_empty[b]), rank);
        continue;
      }
      // the owners have read the sums of the tile before
      if (tile && !__all_sync(0xffffffffu, tc_wait(tc_smem(&sh.sums_empty), (tile - 1) & 1, &sh, p.status, 6))) break;
#pragma unroll 1
      for (int c = 0; c < N; c += 16) {
        if (c >= p.tokens) break;
#pragma unroll
        for (int i = 0; i < G; ++i) {
          float v[16];
          few_ld16(addr + i * N + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c + j >= p.tokens) break;
            const int owner = (c + j) / share, col = c + j - owner * share;
            few_store(tc_mapa(sums, owner) + ((((int)rank * G + i) * share + col) * kRows + lanes + lane) * 4, v[j]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) tc_bar_arrive_remote(tc_smem(&sh.acc_empty[b]), rank);
      if (lane < S) few_arrive(tc_smem(&sh.sums_full), lane);
      if (!__all_sync(0xffffffffu, tc_wait(tc_smem(&sh.sums_full), tile & 1, &sh, p.status, 7))) break;
      asm volatile("fence.acq_rel.cluster;" ::: "memory");
      const int first = (int)rank * share, last = min(min(first + share, N), p.tokens);  // owned columns
      const auto sum = [&](int i, int col) {
        float v = 0.f;
        for (int q = 0; q < S; ++q) v += mine[((q * G + i) * share + col) * kRows + lanes + lane];
        return v;
      };
      if (last - first <= 4) {
        for (int c = first; c < last; ++c) few_put<ACT>(p, g, row0, c, sum(0, c - first), sum(G - 1, c - first));
      } else {
        for (int c = first; c < last; c += 16) {
          float v[G][16];
#pragma unroll
          for (int i = 0; i < G; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] = c + j < last ? sum(i, c + j - first) : 0.f;
          few_put16<ACT>(p, g, row0, c, min(last - c, 16), v[0], v[G - 1]);
        }
      }
      __syncwarp();
      if (lane < S) few_arrive(tc_smem(&sh.sums_empty), lane);
    }
  }

  // teardown
  if (warp == 0 && lane == 0 && sh.give_up) {
    // copies of this CTA may be in flight: wait, bounded, for what was issued
    const uint32_t first = issued > (uint32_t)nstages ? issued - nstages : 0;
    for (uint32_t i = first; i < issued; ++i)
      for (int tries = 0; tries < 64 && !tc_bar_try(tc_smem(&sh.full[i % nstages]), (i / nstages) & 1); ++tries) {
      }
    __nanosleep(1000000);
  }
  tc_fence_before();
  __syncthreads();
  tc_cluster_sync();
  tc_fence_after();
  if (warp == 2) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// Clusters of `split` CTAs the GPU holds at a time, one CTA a SM: clusters
// lie within a group of SMs, so that larger ones leave some over.  Nine tenths of
// the SMs are an estimate: of 3 to 8 CTAs it says 45, 34, 27, 22, 19 and 17 on
// 152 SMs, the occupancy calculator 46, 36, 28, 23, 15 and 15.  The two to four
// too many of 7 and 8 wait for a place (clusters do not wait for one another), so
// that 16 to 19 tiles split so many ways run in two waves where one was counted.
int resident(int split) {
  int ctas = device_sms();
  if (max_ctas_cap() > 0 && max_ctas_cap() < ctas) ctas = max_ctas_cap();
  if (split <= 2) return ctas / split;
  return ctas * 9 / 10 / split;
}

template <int N, int ACT>
cudaError_t few_go(Mx4Args& p, cudaStream_t s, int* grid_out) {
  using F = Few<N, (ACT >= 0)>;
  // the split whose slowest CTA has the fewest K tiles; a sum through the
  // cluster costs about what 4 + columns / 8 stages do (1024 x 2 x 704 row-
  // parallel, 6 K tiles: split 6 ways 5.5 us for 16 tokens and 15.7 for 128,
  // unsplit 4.8 and 6.3; 5120 x 8 x 1728, 56 K tiles: 13.9 split 3 ways)
  int best = 1;
  long long least = -1;
  for (int split = 1; split <= kMaxSplit; ++split) {
    if (split > p.kblocks || resident(split) < 1 || F::stages(split) < 3) break;
    const long long waves = (p.tiles + resident(split) - 1) / resident(split);
    const long long cost = waves * ((p.kblocks + split - 1) / split + (split > 1 ? 4 + F::G * N / 8 : 0));
    if (least < 0 || cost < least) {
      least = cost;
      best = split;
    }
  }
  p.split = best;
  p.stages = F::stages(best);
  const int clusters = p.tiles < resident(best) ? p.tiles : resident(best);
  constexpr auto kern = mx4_few_kernel<N, ACT>;
  const cudaError_t attr = raise_smem<kern>(kMost);
  if (attr != cudaSuccess) return attr;
  *grid_out = clusters * best;
  note_grid(*grid_out);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * best));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = kMost;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)best;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int N>
cudaError_t few_act(Mx4Args& p, bool gated, cudaStream_t s, int* grid) {
  if (!gated) return few_go<N, -1>(p, s, grid);
  if constexpr (N > 64)
    return cudaErrorInvalidValue;  // mx4_few_most
  else
    return p.act == RRA_ACT_SILU ? few_go<N, RRA_ACT_SILU>(p, s, grid) : few_go<N, RRA_ACT_GELU_TANH>(p, s, grid);
}

}  // namespace

// Both kernels, us in a graph, this one first (2070 MHz, 152 SMs):
//                                  tokens   16         32         64        100        128
//   131072 x 5120                       61 / 80    61 / 73    59 / 66    62 / 68    63 / 69
//   50021 x 515 (3 shards)             8.3 / 16   9.4 / 16    11 / 16    14 / 17    14 / 17
//   5120 x 13824 row-parallel           14 / 22    15 / 22    19 / 23    25 / 23    26 / 24
//   1024 x 1408 row-parallel           4.8 / 6.0  4.9 / 6.0  5.4 / 6.2  6.2 / 6.7  6.3 / 7.0
//   gated 13824 rows of K 5120          16 / 25    18 / 24    20 / 21    24 / 21    25 / 21
//   gated 1408 rows of K 1024          5.5 / 6.5  6.6 / 6.5  8.9 / 6.5   13 / 6.6   14 / 6.7
// and gated 13824 rows for 33 tokens 18 / 29, 48 tokens 19 / 22.
// The rule knows the weight rows, not K nor the SM budget: it leaves 5 to 10% for
// gated 13824 rows at 64 tokens and 1024 x 1408 row-parallel at 100 and 128,
// which it gives to the other kernel.
size_t mx4_few_most(size_t rows, bool gated) {
  const size_t bands = rows / kRows, sms = (size_t)device_sms();
  return gated ? (bands < sms / 2 ? 32 : 48) : bands < sms ? 64 : 128;
}

int mx4_few_tile(size_t tokens) { return tokens <= 16 ? 16 : tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128; }

cudaError_t launch_mx4_few(Mx4Args& p, bool gated, cudaStream_t s, int* grid) {
  switch (mx4_few_tile((size_t)p.tokens)) {
    case 16: return few_act<16>(p, gated, s, grid);
    case 32: return few_act<32>(p, gated, s, grid);
    case 64: return few_act<64>(p, gated, s, grid);
    default: return few_act<128>(p, gated, s, grid);
  }
}

}  // namespace rra
