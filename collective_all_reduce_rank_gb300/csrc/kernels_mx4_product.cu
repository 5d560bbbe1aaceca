// kernels_mx4_product.cu -- products of MX4 matrices for more than a few
// tokens: C[t][n] = sum_k X[t][k] W[n][k], both operands as 4-bit codes with a
// scale per 32 columns, multiplied exactly and summed in float32 by the block-
// scaled tensor-core product; column-parallel (a group per rank's shard),
// row-parallel (the ranks' K axes as segments of one: the all-reduce is the
// accumulation), or gated (act(x G^T) * (x U^T) written in MX4 again).
//
// Shape.  A cluster of two CTAs works on a tile of 256 tokens x 256 weight rows
// with tcgen05.mma.cta_group::2, CTA c holding tokens [128c, 128c + 128) of it
// in its tensor memory.  A stage is 256 columns of K: 128 bytes of codes a row
// (one swizzled row), and two scale tiles per 128 rows, which go
// through shared to tensor memory ahead of the stage's four products.
//
// Tensor memory.  Two accumulators of 256 columns and three stages' scales of 24
// do not fit in 512.  The second accumulator starts at column 184, so the two
// share 72 columns: the epilogue reads those of a tile first and then lets the
// next tile's products begin, under the rest of its own work.
//
// Scales.  The tensor cores can copy scales to tensor memory themselves, in
// line with their products, but each of the six copies a stage then cost them
// some 50 cycles (4096 x 5120 x 8 x 1728 gated 256 us, with none of them 190):
// four warps read them from shared memory instead and write them up to three
// stages ahead (gated 238 us with two stages, row-parallel 117 against 107).
// Halves of a stage, five at a time, took 279: the issuing thread then waits and
// commits twice as often.
//
// Roles (16 warps): warps 0 and 3 load X and W, warp 1 of the first CTA issues,
// warp 2 owns the tensor memory, warps 4-11 are the epilogue, 12-15 write
// scales.
#include "act.cuh"
#include "mx4_mma.cuh"

namespace rra {

namespace {

constexpr int kCodes = 128 * 128;  // codes of 128 rows
constexpr int kScalesX = 1024;     // two tiles: a CTA's 128 tokens
constexpr int kScalesW = 2048;     // four: all 256 weight rows
constexpr int kStageBytes = 2 * kCodes + kScalesX + kScalesW;
constexpr int kStages = 5;
constexpr int kSmem = kStages * kStageBytes + kTcEpiWarps * kTcStoreBytes + 1024;
constexpr int kThreads = kTcThreads + 128;
constexpr uint32_t kSecond = 184;  // first column of the second accumulator
constexpr uint32_t kScales = 440;  // first column of the scales: per stage 8 for X and 16 for W
constexpr int kSlots = 3;          // stages whose scales tensor memory holds
static_assert(kStageBytes % 1024 == 0, "a swizzled tile starts on 1024 bytes");
static_assert(kStages <= kTcMaxStages, "barriers");

struct Unit {
  int group, m, n;
};

struct ProductShared : TcShared {
  alignas(8) uint64_t scales_in[kStages];  // this CTA's scales of the stage are in shared memory
};

__device__ __forceinline__ Unit unit_of(const Mx4Args& p, int t) {
  Unit u;
  int g = 0;
  while (g + 1 < p.ngroups && t >= p.group[g + 1].tile0 * p.mt) ++g;
  u.group = g;
  tc_walk(t - p.group[g].tile0 * p.mt, p.mt, p.group[g].tiles, u.m, u.n);
  return u;
}

// 64 columns c0.. of 32 rows from row0 on, stored.
__device__ __forceinline__ void store_pair(const Mx4Args& p, const Mx4Group& g, int row0, int c0, const float* a,
                                           const float* b, uint8_t* buf) {
  const int rows = p.tokens - row0, valid = g.rows - c0;
  if (valid <= 0 || rows <= 0) return;
  if (p.f32) {
    float* o = static_cast<float*>(g.out) + (long long)row0 * g.ld + c0;
    tc_store_f32(buf, a, o, g.ld, rows, valid, g.vec, false);
    if (valid > 32) tc_store_f32(buf, b, o + 32, g.ld, rows, valid - 32, g.vec, false);
  } else {
    tc_stage_bf16(buf, a, 0);
    tc_stage_bf16(buf, b, 4);
    tc_flush_bf16(buf, static_cast<__nv_bfloat16*>(g.out) + (long long)row0 * g.ld + c0, g.ld, rows, valid, g.vec,
                  false);
  }
}

// An epilogue warp's share of a tile: 32 tokens from row0 on, the 128 columns
// of `half`.  The 96 of them nearest its end (LAST) or its start hold all that
// it has of the shared columns: they are read first, and drained() is called.
template <bool LAST, class Drained>
__device__ __forceinline__ void store_tile(const Mx4Args& p, const Unit& u, int row0, int half, uint32_t addr,
                                           uint8_t* buf, Drained drained) {
  const Mx4Group& g = p.group[u.group];
  const int c0 = u.n * 256 + half * 128;
  constexpr int kFirst = LAST ? 64 : 0, kThird = LAST ? 32 : 64, kOther = LAST ? 0 : 96;
  addr += half * 128;
  float a[32], b[32], c[32];
  tc_ld32(addr + kFirst, a);
  tc_ld32(addr + kFirst + 32, b);
  tc_ld32(addr + kThird, c);
  tc_ld_ready(a);
  tc_ld_ready(b);
  tc_ld_ready(c);
  drained();
  store_pair(p, g, row0, c0 + kFirst, a, b, buf);
  tc_ld32(addr + kOther, a);
  tc_ld_ready(a);
  store_pair(p, g, row0, c0 + 64 - kFirst, LAST ? a : c, LAST ? c : a, buf);
}

// Gated: 64 columns of each projection.  What this warp has of the shared
// columns is of the one that comes first, which is read whole.
template <int ACT, bool UP_FIRST, class Drained>
__device__ __forceinline__ void store_gated(const Mx4Args& p, const Unit& u, int row0, int half, uint32_t addr,
                                            Drained drained) {
  const Mx4Group& g = p.group[u.group];
  const int row = row0 + (threadIdx.x & 31);
  float e[2][32];
#pragma unroll
  for (int i = 0; i < 2; ++i) tc_ld32(addr + (UP_FIRST ? 128 : 0) + half * 64 + 32 * i, e[i]);
#pragma unroll
  for (int i = 0; i < 2; ++i) tc_ld_ready(e[i]);
  drained();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = half * 64 + 32 * i;
    float l[32];
    tc_ld32(addr + (UP_FIRST ? 0 : 128) + c, l);
    tc_ld_ready(l);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float unused;
      const float a = UP_FIRST ? l[j] : e[i][j], b = UP_FIRST ? e[i][j] : l[j];
      e[i][j] = a * gate_sigma<ACT>(a, &unused) * b;
    }
    const int c0 = u.n * 128 + c;
    if (row < p.tokens)
      mx4_put_row(e[i], g.rows - c0, static_cast<uint8_t*>(g.out) + (long long)row * g.ld + c0 / 2,
                  g.out_scales + mx_scale_at((size_t)row, (size_t)(c0 / 32), (size_t)g.across));
  }
}

// ACT < 0: a plain product.
template <int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx4_product_kernel(const __grid_constant__ Mx4Args p) {
  constexpr bool GATED = ACT >= 0;
  extern __shared__ uint8_t raw[];
  __shared__ ProductShared sh;
  const uint32_t ring = (tc_smem(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc_cta_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int total = p.tiles * p.mt;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc_bar_init(tc_smem(&sh.full[s]), 1 + 2 * 4);  // codes announced, scales set by four warps a CTA
      tc_bar_init(tc_smem(&sh.empty[s]), 1);
      tc_bar_init(tc_smem(&sh.scales_in[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc_bar_init(tc_smem(&sh.acc_full[b]), 1);
      tc_bar_init(tc_smem(&sh.acc_empty[b]), 2 * kTcEpiWarps);
    }
    sh.give_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(&sh.tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  pdl_next();

  // a stage: codes of W's half, of X's half, scales of X's half, of all of W
  uint32_t issued = 0;
  if (warp == 0 || warp == 3) {
    const bool is_x = warp == 0;
    if (lane == 0) {
      const uint32_t full0 = tc_smem(&sh.full[0]), empty0 = tc_smem(&sh.empty[0]);
      const uint32_t lead0 = tc_mapa(full0, 0);
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
      for (int t = cluster; t < total && ok; t += clusters) {
        const Unit u = unit_of(p, t);
        const int w0 = p.group[u.group].w;
        const int x0 = u.m * 256 + (int)rank * 128;  // first token of this CTA
        // first weight row of this CTA's half: half a tile, or the tile's rows of the gate or the up projection
        const int n0 = GATED ? u.n * 128 : u.n * 256 + (int)rank * 128;
        int seg = 0;
        for (int k = 0; k < p.kblocks; ++k, ++issued) {
          while (seg + 1 < p.nsegs && k >= p.seg_k0[seg + 1]) ++seg;
          const int kk = k - p.seg_k0[seg];
          const int w = (p.nsegs > 1 ? seg : w0);
          if (!tc_wait(empty0 + 8 * s, parity, &sh, p.status, 1)) {
            ok = false;
            break;
          }
          const uint32_t at = ring + s * kStageBytes, bar = lead0 + 8 * s, scales = at + 2 * kCodes;
          const uint32_t mine = tc_smem(&sh.scales_in[s]);
          if (is_x) {
            if (rank == 0) tc_bar_expect(full0 + 8 * s, 4 * kCodes);
            tc_bar_expect(mine, kScalesX + kScalesW);
            tc_tma_load(&p.x[seg], at + kCodes, bar, kk * 128, x0);
            mx4_load(&p.xs[seg], scales, mine, kk * 256, x0 / 128);
            if (GATED) {
              mx4_load(&p.ws[w], scales + kScalesX, mine, kk * 256, u.n);
              mx4_load(&p.ws[w + 1], scales + kScalesX + 1024, mine, kk * 256, u.n);
            } else {
              mx4_load(&p.ws[w], scales + kScalesX, mine, kk * 256, u.n * 2);
            }
          } else {
            tc_tma_load(&p.w[GATED ? w + (int)rank : w], at, bar, kk * 128, n0);
          }
          if (++s == kStages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
      // none of a pair leaves before the last stage releases have landed in it
      for (int i = 0; i < kStages && ok && !is_x; ++i) {
        ok = tc_wait(empty0 + 8 * s, parity, &sh, p.status, 5);
        if (++s == kStages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      uint32_t tile = 0, round = 0;
      int s = 0, slot = 0;
      bool ok = true;
      for (int t = cluster; t < total && ok; t += clusters, ++tile) {
        const uint32_t d = tmem + (tile & 1) * kSecond;
        // the tile before has been read where this one's accumulator begins or ends
        if (tile && !tc_wait(tc_smem(&sh.acc_empty[0]), (tile - 1) & 1, &sh, p.status, 2)) break;
        tc_fence_after();
        for (int k = 0; k < p.kblocks; ++k) {
          if (!tc_wait(tc_smem(&sh.full[s]), round & 1, &sh, p.status, 3)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sw = ring + s * kStageBytes, sx = sw + kCodes;
          const uint32_t tx = tmem + kScales + 24 * slot, tw = tx + 8;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx4_mma<true>(d, tc_desc<false>(sx + 32 * i), tc_desc<false>(sw + 32 * i), mx4_idesc(256, 256, 2 * (i & 1)),
                          tx + 4 * (i >> 1), tw + 8 * (i >> 1), (uint32_t)(k > 0 || i > 0));
          if (++slot == kSlots) slot = 0;
          tc_commit(tc_smem(&sh.empty[s]));
          if (++s == kStages) {
            s = 0;
            ++round;
          }
        }
        if (ok) tc_commit(tc_smem(&sh.acc_full[tile & 1]));
      }
    }
    __syncwarp();
  } else if (warp >= 12) {
    // this quarter of the lanes' scales
    const uint32_t lanes = tmem + kScales + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t stage = 0, round = 0, round_before = 0;
    int s = 0, before = 0;  // places of this stage and of the one kSlots stages ago
    int slot = 0;
    bool ok = true;
    for (int t = cluster; t < total && ok; t += clusters)
      for (int k = 0; k < p.kblocks; ++k, ++stage) {
        ok = tc_wait(tc_smem(&sh.scales_in[s]), round & 1, &sh, p.status, 8);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint4* from = reinterpret_cast<const uint4*>(raw + (ring - tc_smem(raw)) + s * kStageBytes + 2 * kCodes);
        const uint4 x0 = from[lane], x1 = from[32 + lane], a0 = from[64 + lane], a1 = from[96 + lane];
        const uint4 b0 = from[128 + lane], b1 = from[160 + lane];
        // the products of kSlots stages ago no longer read these columns
        if (stage >= kSlots) {
          ok = tc_wait(tc_smem(&sh.empty[before]), round_before & 1, &sh, p.status, 7);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (++before == kStages) {
            before = 0;
            ++round_before;
          }
        }
        const uint32_t to = lanes + 24 * slot;
        mx4_st8(to, x0, x1);
        mx4_st8(to + 8, a0, b0);
        mx4_st8(to + 16, a1, b1);
        mx4_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tc_bar_arrive_remote(tc_smem(&sh.full[s]), 0);
        if (++slot == kSlots) slot = 0;
        if (++s == kStages) {
          s = 0;
          ++round;
        }
      }
  } else if (warp >= 4) {
    const int quad = warp & 3, half = (warp - 4) >> 2;
    uint8_t* buf = raw + (ring - tc_smem(raw)) + kStages * kStageBytes + (warp - 4) * kTcStoreBytes;
    uint32_t tile = 0;
    for (int t = cluster; t < total; t += clusters, ++tile) {
      const uint32_t b = tile & 1;
      if (!__all_sync(0xffffffffu, tc_wait(tc_smem(&sh.acc_full[b]), (tile >> 1) & 1, &sh, p.status, 4))) break;
      tc_fence_after();
      const Unit u = unit_of(p, t);
      // the shared columns are the first accumulator's last, the second's first
      const auto drained = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tc_bar_arrive_remote(tc_smem(&sh.acc_empty[0]), 0);
      };
      const uint32_t addr = tmem + b * kSecond + ((uint32_t)(quad * 32) << 16);
      const int row0 = u.m * 256 + (int)rank * 128 + quad * 32;
      if constexpr (GATED) {
        if (b)
          store_gated<ACT, false>(p, u, row0, half, addr, drained);
        else
          store_gated<ACT, true>(p, u, row0, half, addr, drained);
      } else {
        if (b)
          store_tile<false>(p, u, row0, half, addr, buf, drained);
        else
          store_tile<true>(p, u, row0, half, addr, buf, drained);
      }
    }
  }

  // teardown
  if ((warp == 0 || warp == 3) && lane == 0 && sh.give_up) {
    // copies of this CTA may be in flight: wait, bounded, for what was issued
    const uint32_t first = issued > (uint32_t)kStages ? issued - kStages : 0;
    for (uint32_t i = first; i < issued; ++i)
      for (int tries = 0; tries < 64 && !tc_bar_try(tc_smem(&sh.full[i % kStages]), (i / kStages) & 1); ++tries) {
      }
    __nanosleep(1000000);
  }
  tc_fence_before();
  __syncthreads();
  tc_cluster_sync();
  tc_fence_after();
  if (warp == 2) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <int ACT>
cudaError_t go(const Mx4Args& p, cudaStream_t s, int* grid_out) {
  constexpr auto kern = mx4_product_kernel<ACT>;
  const cudaError_t attr = raise_smem<kern>(kSmem);
  if (attr != cudaSuccess) return attr;
  const int grid = 2 * tc_clusters(p.tiles * p.mt);
  if (grid_out) *grid_out = grid;
  return launch_pdl(kern, grid, kThreads, kSmem, s, p);
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Args& p, bool gated, cudaStream_t s, int* grid) {
  if (!gated) return go<-1>(p, s, grid);
  return p.act == RRA_ACT_SILU ? go<RRA_ACT_SILU>(p, s, grid) : go<RRA_ACT_GELU_TANH>(p, s, grid);
}

}  // namespace rra
