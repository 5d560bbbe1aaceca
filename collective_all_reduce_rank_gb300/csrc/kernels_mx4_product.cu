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
// Tensor memory.  Two accumulators of 256 columns and four stages' scales of 24
// do not fit in 512.  The second accumulator starts at column 160, so the two
// share 96 columns: the epilogue reads those of a tile first and then lets the
// next tile's products begin, under the rest of its own work.
//
// Scales.  The tensor cores can copy scales to tensor memory themselves, in
// line with their products, but each of the six copies a stage then cost them
// some 50 cycles (4096 x 5120 x 8 x 1728 gated 256 us, with none of them 190):
// four warps read them from shared memory instead and write them up to four
// stages ahead (two measured 15 us slower), announced on the barrier of the
// stage's codes (a barrier of their own 25 us: what the issuing thread waits for
// and commits is on the way of every product).
//
// Roles (16 warps): warps 0 and 3 load X and W, warp 2 their scales (it also owns
// the tensor memory), warp 1 of the first CTA issues, warps 4-11 are the
// epilogue, 12-15 write scales.
#include "act.cuh"
#include "mx4_mma.cuh"

namespace rra {

namespace {

constexpr int kCodes = 128 * 128;  // codes of 128 rows
constexpr int kScalesX = 1024;     // two tiles: a CTA's 128 tokens
constexpr int kScalesW = 2048;     // four: all 256 weight rows
constexpr int kScaleBytes = kScalesX + kScalesW;
constexpr int kScaleStages = 6;
constexpr int kThreads = kTcThreads + 128;
constexpr uint32_t kSecond = 160;  // first column of the second accumulator
constexpr uint32_t kScales = 416;  // first column of the scales: per stage 8 for X and 16 for W
constexpr int kSlots = 4;          // stages whose scales tensor memory holds

// Shared memory: a ring of codes (W's half, X's half), one of scales, and, for
// plain products, the epilogue's staging.
template <bool GATED>
struct Layout {
  static constexpr int kStages = GATED ? 6 : 5;
  static constexpr int kStore = kStages * 2 * kCodes + kScaleStages * kScaleBytes;
  static constexpr int kBytes = kStore + (GATED ? 0 : kTcEpiWarps * kTcStoreBytes) + 1024;
  static_assert(kBytes + 1024 <= 227 * 1024, "shared memory of a CTA, with what is static");
};

struct Unit {
  int group, m, n;
};

struct ProductShared : TcShared {
  alignas(8) uint64_t scales_in[kScaleStages];  // this CTA's scales of a stage are in shared memory
  alignas(8) uint64_t scales_out[kScaleStages];  // its four warps have read them
};

__device__ __forceinline__ Unit unit_of(const Mx4Args& p, int t) {
  Unit u;
  int g = 0;
  while (g + 1 < p.ngroups && t >= p.group[g + 1].tile0 * p.mt) ++g;
  u.group = g;
  tc_walk(t - p.group[g].tile0 * p.mt, p.mt, p.group[g].tiles, u.m, u.n);
  return u;
}

// Blocks of whole 64 bfloat16 or 32 float32 columns from a warp's staging
// buffer, without a branch in the way of the loads and stores.  With those of
// tc_epilogue.cuh, which any block can take, 333 x 515 x 50021 takes 30.5 us
// (float32 59), 512 tokens of the feed-forward block 63; with these 25.8 (30) and
// 58.
// VEC: rows of whole 16-byte units, four a step.
__device__ __forceinline__ void put_vec(const uint8_t* buf, char* dst, long long row_bytes, int rows) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  __syncwarp();
  uint4 u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    u[i] = *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
  }
  dst += (lane >> 3) * row_bytes + 16 * c;
#pragma unroll
  for (int i = 0; i < 8; ++i, dst += 4 * row_bytes)
    if (4 * i + (lane >> 3) < rows) *reinterpret_cast<uint4*>(dst) = u[i];
  __syncwarp();
}

// Rows of whole words: one a step.
__device__ __forceinline__ void put_words(const uint8_t* buf, char* dst, long long row_bytes, int rows) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  dst += 4 * lane;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 16) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i] = *reinterpret_cast<const uint32_t*>(buf + (r0 + i) * 128 + (((lane >> 2) ^ (i & 7)) << 4) + 4 * (lane & 3));
#pragma unroll
    for (int i = 0; i < 16; ++i, dst += row_bytes)
      if (r0 + i < rows) *reinterpret_cast<uint32_t*>(dst) = w[i];
  }
  __syncwarp();
}

// Rows of 64 bfloat16 that start on any of them: one that starts in the middle
// of a word is stored as its 31 whole words; the columns at its ends, `first`
// and `last` of the lane's row, are stored for all rows at once (333 x 512 x
// 50021 33 us with tc_epilogue.cuh's stores, 30 with these, 59 with the ends
// stored row by row).
__device__ __forceinline__ void put_halves(const uint8_t* buf, __nv_bfloat16* o, long long ld, int rows, float first,
                                           float last) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  __nv_bfloat16* own = o + lane * ld;
  const bool ends = lane < rows && ((uintptr_t)own & 2);
  if (ends) own[0] = __float2bfloat16_rn(first);
  if (ends) own[63] = __float2bfloat16_rn(last);
  char* dst = reinterpret_cast<char*>(o) + 4 * lane;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 16) {
    uint32_t w[16], next[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i] = *reinterpret_cast<const uint32_t*>(buf + (r0 + i) * 128 + (((lane >> 2) ^ (i & 7)) << 4) + 4 * (lane & 3));
#pragma unroll
    for (int i = 0; i < 16; ++i) next[i] = __shfl_down_sync(0xffffffffu, w[i], 1);
#pragma unroll
    for (int i = 0; i < 16; ++i, dst += 2 * ld) {
      const uint32_t off = (uint32_t)(uintptr_t)dst & 2;
      if (r0 + i < rows && lane < 32 - (int)(off / 2))
        *reinterpret_cast<uint32_t*>(dst + off) = __funnelshift_r(w[i], next[i], 8 * off);
    }
  }
  __syncwarp();
}

// A row's 32 float32 into the staging buffer.
__device__ __forceinline__ void stage_f32(uint8_t* buf, const float* v) {
  const int r = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(buf + r * 128 + ((c ^ (r & 7)) << 4)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

// 64 columns c0.. of 32 rows from row0 on, stored.
__device__ __forceinline__ void store_pair(const Mx4Args& p, const Mx4Group& g, int row0, int c0, const float* a,
                                           const float* b, uint8_t* buf) {
  const int rows = p.tokens - row0, valid = g.rows - c0;
  if (valid <= 0 || rows <= 0) return;
  const bool whole = valid >= 64;
  if (p.f32) {
    float* o = static_cast<float*>(g.out) + (long long)row0 * g.ld + c0;
    if (whole) {
      char* dst = reinterpret_cast<char*>(o);
      stage_f32(buf, a);
      g.vec ? put_vec(buf, dst, g.ld * 4, rows) : put_words(buf, dst, g.ld * 4, rows);
      stage_f32(buf, b);
      g.vec ? put_vec(buf, dst + 128, g.ld * 4, rows) : put_words(buf, dst + 128, g.ld * 4, rows);
      return;
    }
    tc_store_f32(buf, a, o, g.ld, rows, valid, g.vec, false);
    if (valid > 32) tc_store_f32(buf, b, o + 32, g.ld, rows, valid - 32, g.vec, false);
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g.out) + (long long)row0 * g.ld + c0;
    tc_stage_bf16(buf, a, 0);
    tc_stage_bf16(buf, b, 4);
    if (whole && g.vec)
      put_vec(buf, reinterpret_cast<char*>(o), g.ld * 2, rows);
    else if (whole && g.ld % 2 == 0 && ((uintptr_t)o & 3) == 0)
      put_words(buf, reinterpret_cast<char*>(o), g.ld * 2, rows);
    else if (whole)
      put_halves(buf, o, g.ld, rows, a[0], b[31]);
    else
      tc_flush_bf16(buf, o, g.ld, rows, valid, g.vec, false);
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
  constexpr int nstages = Layout<GATED>::kStages;
  constexpr uint32_t stage_bytes = 2 * kCodes, wbytes = kCodes;  // a stage of codes: W's half, then X's
  const uint32_t scale_ring = ring + nstages * stage_bytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < nstages; ++s) {
      tc_bar_init(tc_smem(&sh.full[s]), 1 + 2 * 4);  // codes announced, scales set by four warps a CTA
      tc_bar_init(tc_smem(&sh.empty[s]), 1);
    }
    for (int s = 0; s < kScaleStages; ++s) {
      tc_bar_init(tc_smem(&sh.scales_in[s]), 1);
      tc_bar_init(tc_smem(&sh.scales_out[s]), 4);
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
        // first token of this CTA; first weight row of its half: half a tile, or the tile's rows of the gate or the up
        // projection
        const int x0 = u.m * 256 + (int)rank * 128;
        const int n0 = GATED ? u.n * 128 : u.n * 256 + (int)rank * 128;
        int seg = 0;
        for (int k = 0; k < p.kblocks; ++k, ++issued) {
          while (seg + 1 < p.nsegs && k >= p.seg_k0[seg + 1]) ++seg;
          const int kk = k - p.seg_k0[seg];
          const int w = p.nsegs > 1 ? seg : w0;
          if (!tc_wait(empty0 + 8 * s, parity, &sh, p.status, 1)) {
            ok = false;
            break;
          }
          const uint32_t at = ring + s * stage_bytes, bar = lead0 + 8 * s;
          if (is_x) {
            if (rank == 0) tc_bar_expect(full0 + 8 * s, 2 * stage_bytes);
            tc_tma_load(&p.x[seg], at + wbytes, bar, kk * 128, x0);
          } else {
            tc_tma_load(&p.w[GATED ? w + (int)rank : w], at, bar, kk * 128, n0);
          }
          if (++s == nstages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
      // none of a pair leaves before the last stage releases have landed in it
      for (int i = 0; i < nstages && ok && !is_x; ++i) {
        ok = tc_wait(empty0 + 8 * s, parity, &sh, p.status, 5);
        if (++s == nstages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // scales, in a ring of their own: they are small, and are asked for further
    // ahead than codes can be
    if (lane == 0) {
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
      for (int t = cluster; t < total && ok; t += clusters) {
        const Unit u = unit_of(p, t);
        const int w0 = p.group[u.group].w, band = u.m * 2 + (int)rank;
        int seg = 0;
        for (int k = 0; k < p.kblocks; ++k) {
          while (seg + 1 < p.nsegs && k >= p.seg_k0[seg + 1]) ++seg;
          const int at_k = (k - p.seg_k0[seg]) * 256, w = p.nsegs > 1 ? seg : w0;
          if (!tc_wait(tc_smem(&sh.scales_out[s]), parity, &sh, p.status, 6)) {
            ok = false;
            break;
          }
          const uint32_t at = scale_ring + s * kScaleBytes, bar = tc_smem(&sh.scales_in[s]);
          tc_bar_expect(bar, kScaleBytes);
          mx4_load(&p.xs[seg], at, bar, at_k, band);
          if (GATED) {
            mx4_load(&p.ws[w], at + kScalesX, bar, at_k, u.n);
            mx4_load(&p.ws[w + 1], at + kScalesX + 1024, bar, at_k, u.n);
          } else {
            mx4_load(&p.ws[w], at + kScalesX, bar, at_k, u.n * 2);
          }
          if (++s == kScaleStages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // The whole warp walks the stages and one lane of it issues, so that what an
    // instruction takes is computed once a warp, in uniform registers (by a lane
    // of its own a product took 90 cycles to issue, a stage 750).
    if (rank == 0) {
      const bool lead = mx4_elect();
      constexpr uint32_t idesc = mx4_idesc(256, 256);
      uint32_t tile = 0, round = 0;
      int s = 0, slot = 0;
      bool ok = true;
      for (int t = cluster; t < total && ok; t += clusters, ++tile) {
        const uint32_t d = tmem + (tile & 1) * kSecond;
        // the tile before has been read where this one's accumulator begins or ends
        if (tile) {
          ok = __all_sync(0xffffffffu, tc_wait(tc_smem(&sh.acc_empty[0]), (tile - 1) & 1, &sh, p.status, 2));
          if (!ok) break;
        }
        tc_fence_after();
        for (int k = 0; k < p.kblocks; ++k) {
          ok = __all_sync(0xffffffffu, tc_wait(tc_smem(&sh.full[s]), round & 1, &sh, p.status, 3));
          if (!ok) break;
          tc_fence_after();
          const uint32_t sw = ring + s * stage_bytes, sx = sw + wbytes;
          const uint32_t tx = tmem + kScales + 24 * slot, tw = tx + 8;
          if (lead) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx4_mma<true>(d, tc_desc<false>(sx + 32 * i), tc_desc<false>(sw + 32 * i),
                            idesc | mx4_idesc_scales(2 * (i & 1)), tx + 4 * (i >> 1), tw + 8 * (i >> 1),
                            (uint32_t)(k > 0 || i > 0));
            tc_commit(tc_smem(&sh.empty[s]));
          }
          __syncwarp();
          if (++slot == kSlots) slot = 0;
          if (++s == nstages) {
            s = 0;
            ++round;
          }
        }
        if (ok && lead) tc_commit(tc_smem(&sh.acc_full[tile & 1]));
        __syncwarp();
      }
    }
    __syncwarp();
  } else if (warp >= 12) {
    // this quarter of the lanes' scales
    const uint32_t lanes = tmem + kScales + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t n = cluster < total ? (uint32_t)((total - cluster + clusters - 1) / clusters) * p.kblocks : 0;
    uint32_t round = 0, round_before = 0;
    int from = 0;           // place in the ring of scales
    int s = 0, before = 0;  // places in that of codes, of this stage and of the one kSlots stages ago
    int slot = 0;
    for (uint32_t stage = 0; stage < n; ++stage) {
      bool ok = tc_wait(tc_smem(&sh.scales_in[from]), round & 1, &sh, p.status, 8);
      const uint4* at = reinterpret_cast<const uint4*>(raw + (scale_ring - tc_smem(raw)) + from * kScaleBytes) + lane;
      const uint4 x0 = at[0], x1 = at[32], a0 = at[64], a1 = at[96], b0 = at[128], b1 = at[160];
      // the products of kSlots stages ago no longer read these columns
      if (stage >= kSlots) {
        ok = ok && tc_wait(tc_smem(&sh.empty[before]), round_before & 1, &sh, p.status, 7);
        if (++before == nstages) {
          before = 0;
          ++round_before;
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t to = lanes + 24 * slot;
      mx4_st8(to, x0, x1);
      mx4_st8(to + 8, a0, b0);
      mx4_st8(to + 16, a1, b1);
      mx4_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc_bar_arrive_remote(tc_smem(&sh.full[s]), 0);
        tc_bar_arrive_remote(tc_smem(&sh.scales_out[from]), rank);
      }
      if (++from == kScaleStages) {
        from = 0;
        ++round;
      }
      if (++slot == kSlots) slot = 0;
      if (++s == nstages) s = 0;
    }
  } else if (warp >= 4) {
    const int quad = warp & 3, half = (warp - 4) >> 2;
    uint8_t* buf = raw + (ring - tc_smem(raw)) + Layout<GATED>::kStore + (warp - 4) * kTcStoreBytes;
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
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <int ACT>
cudaError_t go(const Mx4Args& p, cudaStream_t s, int* grid_out) {
  constexpr auto kern = mx4_product_kernel<ACT>;
  const cudaError_t attr = raise_smem<kern>(Layout<(ACT >= 0)>::kBytes);
  if (attr != cudaSuccess) return attr;
  const int grid = 2 * tc_clusters(p.tiles * p.mt);
  if (grid_out) *grid_out = grid;
  return launch_pdl(kern, grid, kThreads, Layout<(ACT >= 0)>::kBytes, s, p);
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Args& p, bool gated, cudaStream_t s, int* grid) {
  if (!gated) return go<-1>(p, s, grid);
  return p.act == RRA_ACT_SILU ? go<RRA_ACT_SILU>(p, s, grid) : go<RRA_ACT_GELU_TANH>(p, s, grid);
}

}  // namespace rra
