// tc_gemm.cuh -- the tensor-core product the training operators are built
// on: C[m][n] = sum_k A[m][k] B[n][k] in bfloat16 with float32 accumulators
// in tensor memory, and an epilogue per operator that turns the accumulators
// into what the operator stores, so that neither logits nor projections are
// written to memory.
//
// Bound.  A tile's 64-deep step is 512 cycles of the tensor pipe and moves 64
// KB from L2 to its two SMs, 64 bytes a cycle each, which is about what L2
// gives: both sides are near their limits, and everything else has to stay
// out of the way.  Measured on one GB300 (ncu): tensor pipe 91-96% active in
// all five products of a 2048-token step (hidden 5120).  The clock under the
// power limit then sets the rate: 4096 x 5120 x 4 x 3456 gated backward 2.06-
// 2.13 ms call after call (1.64-1.69 PFLOP/s; 1.78 ms and 1.96 in a few calls
// from a cool start), 2048 x 5120 x 131072 loss 1.56-1.61 ms (1.71-1.76; 1.36
// and 2.02), beside a library bfloat16 product of 8192^3 at 1.70 sustained and
// 1.87 in a burst.
//
// Shape.  A cluster of two CTAs works on a 256 x 256 tile of C with
// tcgen05.mma.cta_group::2: CTA c of the pair holds rows [128c, 128c+128)
// of the tile in its tensor memory, and rows [128c, ...) of A and of B's
// half in shared memory, so each operand byte is staged once per pair (a
// single-CTA 128 x 256 tile would read 1.5x the shared memory per product).
// Both 256-column accumulators of a CTA's 512 tensor-memory columns are
// used: the epilogue of one tile runs under the products of the next.
//
// Roles (12 warps): warps 0 and 3 issue the TMA loads of their CTA's halves
// of A and B into a ring of 64-deep K stages; warp 1 of the first CTA issues
// the products; warp 2 owns the tensor-memory allocation; warps 4-11 are the
// epilogue (warp w reads the 32 lanes of quadrant w % 4 and one half of the
// columns).
//
// Operands are K-major (rows of K contiguous: activations times weights) or
// MN-major (rows of M or N contiguous: the transposed products of a
// backward pass), both in the 128-byte swizzle; TMA writes zeros past every
// extent, so ragged M, N and K need no other handling here.
//
// Waits.  Every mbarrier wait is bounded (kTcWaitNs); a wait that expires
// raises the CTA's give-up flag and records RRA_ERR_TIMEOUT in the status
// word, every role of the CTA leaves its loop, and the teardown waits, again
// bounded, for copies in flight.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pdl.cuh"
#include "rra_internal.h"
#include "smem_limit.h"
#include "tc_host.h"

namespace rra {

constexpr int kTcThreads = 384;
constexpr int kTcEpiWarps = 8;
constexpr int kTcBK = kTcKBlock;
constexpr int kTcHalfBytes = 128 * kTcBK * 2;  // one operand's half tile of a CTA
constexpr int kTcStageBytes = 2 * kTcHalfBytes;
constexpr int kTcStages = 6;      // of full halves; narrower ones fit up to
constexpr int kTcMaxStages = 12;  // this many in the same bytes
constexpr int kTcRingBytes = kTcStages * kTcStageBytes;
constexpr int kTcStoreBytes = 4096;  // store staging of one epilogue warp (tc_epilogue.cuh)
constexpr int kTcSmem = kTcRingBytes + kTcEpiWarps * kTcStoreBytes + 1024;  // + alignment slack
constexpr unsigned long long kTcWaitNs = 2000ull * 1000 * 1000;

// ---------------------------------------------------------------------------
// PTX.  An .aligned instruction needs all lanes of its warp at once: each
// helper that issues one joins the lanes first, since its caller may have
// sent them along different branches (a row's target, a row past the end).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t tc_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t tc_cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void tc_cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ bool tc_bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}

// Arrive on the barrier at the same offset in CTA `cta` of the cluster.  What
// it reports is the end of tensor-memory reads, whose values are in registers
// (tcgen05.wait::ld): no memory needs publishing to the cluster, and a release
// at that scope would wait for the epilogue's global stores.
__device__ __forceinline__ void tc_bar_arrive_remote(uint32_t bar, uint32_t cta) {
  asm volatile(
      "{\n.reg .b32 a;\n"
      "mapa.shared::cluster.u32 a, %0, %1;\n"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n}\n" ::"r"(bar),
      "r"(cta)
      : "memory");
}

__device__ __forceinline__ void tc_bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Address in the cluster's shared window of `addr` in CTA `cta`.
__device__ __forceinline__ uint32_t tc_mapa(uint32_t addr, uint32_t cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}

// TMA tile load into this CTA whose completion counts on `bar`, a cluster
// address: the barrier of the pair's first CTA.
__device__ __forceinline__ void tc_tma_load(const CUtensorMap* map, uint32_t dst, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on the barrier at this offset in both CTAs once every product
// issued so far has finished.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 2^x by the special function unit (two units in the last place, results
// below 2^-126 flushed to zero: nothing beside the 1 of a row's maximum).
__device__ __forceinline__ float tc_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 lanes x 32 columns of float32: lane l of the warp gets row l.
__device__ __forceinline__ void tc_ld32(uint32_t addr, float* v) {
  uint32_t r[32];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Wait for this thread's tensor-memory reads; the values become usable here
// (they are operands, so no use can move above the wait).
__device__ __forceinline__ void tc_ld_ready(float* v) {
  __syncwarp();
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                 "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                 "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]),
                 "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}


// Shared-memory operand descriptor, 128-byte swizzle.  K-major: rows of 128
// bytes, groups of 8 rows 1024 bytes apart (the stride offset; the leading
// offset is unused).  MN-major: 64 elements of M or N per 128-byte row, one
// row per k, groups of 8 k 1024 bytes apart, the next 64 of M or N a box
// (64 rows) further, the leading offset.
template <bool MN>
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr) {
  constexpr uint64_t lbo = MN ? (kTcHalfBytes / 2) >> 4 : 1;
  constexpr uint64_t base = (lbo << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
  return base | (uint64_t)((addr & 0x3FFFF) >> 4);
}

// Instruction descriptor: float32 accumulators, bfloat16 operands, their
// major-ness, N = 256 and M = 256 over the pair.
template <bool AMN, bool BMN>
constexpr uint32_t kTcIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((AMN ? 1u : 0u) << 15) |
                              ((BMN ? 1u : 0u) << 16) | ((256u >> 3) << 17) | ((256u >> 4) << 24);

// ---------------------------------------------------------------------------
// bounded waits
// ---------------------------------------------------------------------------
struct TcShared {
  alignas(8) uint64_t full[kTcMaxStages];
  alignas(8) uint64_t empty[kTcMaxStages];
  alignas(8) uint64_t acc_full[2];
  alignas(8) uint64_t acc_empty[2];
  uint32_t tmem;
  volatile uint32_t give_up;
};

static __device__ __noinline__ bool tc_wait_slow(uint32_t bar, uint32_t parity, TcShared* sh, DevStatus* st, int what) {
  const unsigned long long d = (1ull << 63) | ((unsigned long long)what << 32) | 0xFFFF0000ull | (blockIdx.x & 0xFFFF);
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (uint32_t it = 0; it < (1u << 26); ++it) {
    if (tc_bar_try(bar, parity)) return true;
    if (sh->give_up) return false;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > kTcWaitNs) break;
  }
  sh->give_up = 1;
  atomicCAS(&st->code, 0, (int)RRA_ERR_TIMEOUT);
  atomicCAS(&st->detail, 0ull, d);
  return false;
}

__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, TcShared* sh, DevStatus* st, int what) {
  if (tc_bar_try(bar, parity)) return true;
  return tc_wait_slow(bar, parity, sh, st, what);
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
struct TcTile {
  int group, m, n;
  int slot;    // which part of the split tiles this is (-1: a whole tile)
  int k0, k1;  // K blocks
};

// K blocks of unit t: all of them, or one of the parts of a split tile.
__device__ __forceinline__ void tc_krange(const TcArgs& p, int t, int& k0, int& k1) {
  k0 = 0;
  k1 = p.kblocks;
  if (t >= p.full) {
    const int part = (t - p.full) % p.splits;
    k0 = (int)((long long)p.kblocks * part / p.splits);
    k1 = (int)((long long)p.kblocks * (part + 1) / p.splits);
  }
}

// Where tile u of a group of mt x nt tiles lies: bands of kTcBand tile rows,
// down the band first, so that the tiles running at one time share few rows
// of A and columns of B in L2.
__device__ __forceinline__ void tc_walk(int u, int mt, int nt, int& m, int& n) {
  const int band = u / (kTcBand * nt);
  const int rows = min(kTcBand, mt - band * kTcBand);
  const int v = u - band * kTcBand * nt;
  m = band * kTcBand + v % rows;
  n = v / rows;
}

// Unit t of the launch: whole tiles first, group by group, then the parts of
// the split tiles.
__device__ __forceinline__ TcTile tc_tile(const TcArgs& p, int t) {
  TcTile x;
  tc_krange(p, t, x.k0, x.k1);
  x.slot = t - p.full;
  int u = x.slot < 0 ? t : p.full + x.slot / p.splits;
  int g = 0;
  while (g + 1 < p.ngroups && u >= p.group[g + 1].tile0) ++g;
  x.group = g;
  u -= p.group[g].tile0;
  tc_walk(u, p.group[g].mt, p.group[g].nt, x.m, x.n);
  return x;
}

// ---------------------------------------------------------------------------
// kernel.  Epi::run(p, tile, row0, half, addr, buf, state) consumes one
// accumulator: each lane of a warp row row0 + lane of C and the columns of
// half `half` (0 or 1) of the tile, with kTcStoreBytes of shared memory for
// its stores.  What it needs from memory beside the accumulator can be asked
// for a tile ahead: Epi::ahead issues loads before the tile before is
// consumed, Epi::more those that depend on them, after it.
// ---------------------------------------------------------------------------
struct TcNoState {
  struct State {};
  static __device__ __forceinline__ State ahead(const TcArgs&, const TcTile&, int, int) { return {}; }
  static __device__ __forceinline__ void more(const TcArgs&, const TcTile&, int, int, State&) {}
};

template <bool AMN, bool BMN, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
    tc_gemm_kernel(const __grid_constant__ TcArgs p) {
  extern __shared__ uint8_t raw[];
  __shared__ TcShared sh;
  const uint32_t stages = (tc_smem(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc_cta_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int total = tc_units(p);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.shape.stages; ++s) {
      tc_bar_init(tc_smem(&sh.full[s]), 1);
      tc_bar_init(tc_smem(&sh.empty[s]), 1);
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

  // a stage holds B's half, then A's; an A shorter than 128 rows is read on
  // into the next stage or the store staging behind the ring
  const int nstages = p.shape.stages;
  constexpr uint32_t bbytes = kTcHalfBytes;
  const uint32_t abytes = AMN ? kTcHalfBytes : (uint32_t)p.shape.a_rows * 128;
  const uint32_t stage_bytes = abytes + bbytes;
  uint32_t issued = 0;  // producers: stages loaded so far
  if (warp == 0 || warp == 3) {
    // warp 0 loads A and announces each stage's bytes, warp 3 loads B.  With
    // one thread issuing both, the tensor pipe was 96% active with two boxes a
    // stage, 89% with three and 73% with the four of two MN-major operands
    // (backward of 4096 x 5120 x 4 x 3456: 1.87 ms, with two threads 1.82 ms)
    const bool is_a = warp == 0;
    if (lane == 0 && (!is_a || rank == 0 || AMN || p.shape.a_ctas > 1)) {
      const uint32_t full0 = tc_smem(&sh.full[0]), empty0 = tc_smem(&sh.empty[0]);
      const uint32_t lead0 = tc_mapa(full0, 0);
      const uint32_t dst0 = is_a ? stages + bbytes : stages;
      const uint32_t bytes = 2 * bbytes + (AMN ? 2u : (uint32_t)p.shape.a_ctas) * abytes;
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
      for (int t = cluster; t < total && ok; t += clusters) {
        const TcTile x = tc_tile(p, t);
        const TcGroup& g = p.group[x.group];
        const int mn0 = is_a ? g.m0 + x.m * 256 + (int)rank * 128
                             : g.n0 + (p.pair_b ? x.n * 128 : x.n * 256 + (int)rank * 128);
        int seg = 0;
        for (int k = x.k0; k < x.k1 && ok;) {
          while (seg + 1 < p.nsegs && k >= p.seg_k0[seg + 1]) ++seg;
          const int from = p.seg_k0[seg];
          const int to = seg + 1 < p.nsegs ? min(x.k1, p.seg_k0[seg + 1]) : x.k1;
          const bool own = p.nsegs > 1 && !p.rest_k;  // each segment has its maps
          const CUtensorMap* map = is_a ? &p.a[own ? seg : g.a] : &p.b[own ? seg : (p.pair_b ? g.b + (int)rank : g.b)];
          for (int kk = (k - from) * kTcBK + (is_a && seg ? p.rest_k : 0); k < to; ++k, kk += kTcBK, ++issued) {
            if (!tc_wait(empty0 + 8 * s, parity, &sh, p.status, 1)) {
              ok = false;
              break;
            }
            if (is_a && rank == 0) tc_bar_expect(full0 + 8 * s, bytes);
            const uint32_t dst = dst0 + s * stage_bytes, bar = lead0 + 8 * s;
            if (is_a ? AMN : BMN) {
              tc_tma_load(map, dst, bar, mn0, kk);
              tc_tma_load(map, dst + kTcHalfBytes / 2, bar, mn0 + 64, kk);
            } else {
              tc_tma_load(map, dst, bar, kk, mn0);
            }
            if (++s == nstages) {
              s = 0;
              parity ^= 1;
            }
          }
        }
      }
      // A stage's release is a commit of the first CTA's products that arrives
      // in both CTAs: none may leave before the last ones have landed in it.
      for (int i = 0; i < nstages && ok && !is_a; ++i) {
        ok = tc_wait(empty0 + 8 * s, parity, &sh, p.status, 5);
        if (++s == nstages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      uint32_t tile = 0, round = 0;
      int s = 0;
      bool ok = true;
      for (int t = cluster; t < total && ok; t += clusters) {
        int k0, k1;
        tc_krange(p, t, k0, k1);
        if (k0 == k1) continue;  // a part of a K axis shorter than its parts
        const uint32_t buf = tile & 1, d = tmem + buf * 256;
        if (!tc_wait(tc_smem(&sh.acc_empty[buf]), ((tile >> 1) & 1) ^ 1, &sh, p.status, 2)) break;
        tc_fence_after();
        for (int k = k0; k < k1; ++k) {
          if (!tc_wait(tc_smem(&sh.full[s]), round & 1, &sh, p.status, 3)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sb = stages + s * stage_bytes, sa = sb + bbytes;
#pragma unroll
          for (int i = 0; i < kTcBK / 16; ++i)
            tc_mma(d, tc_desc<AMN>(sa + i * (AMN ? 2048 : 32)), tc_desc<BMN>(sb + i * (BMN ? 2048 : 32)),
                   kTcIdesc<AMN, BMN>, (uint32_t)(k > k0 || i > 0));
          tc_commit(tc_smem(&sh.empty[s]));
          if (++s == nstages) {
            s = 0;
            ++round;
          }
        }
        if (ok) tc_commit(tc_smem(&sh.acc_full[buf]));
        ++tile;
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int row_in = (int)rank * 128 + quad * 32;
    uint32_t tile = 0;
    TcTile next{};
    typename Epi::State state, after;
    if (cluster < total) {
      next = tc_tile(p, cluster);
      after = Epi::ahead(p, next, next.m * 256 + row_in, half);
      Epi::more(p, next, next.m * 256 + row_in, half, after);
    }
    for (int t = cluster; t < total; t += clusters) {
      const TcTile x = next;
      state = after;
      if (t + clusters < total) {
        next = tc_tile(p, t + clusters);
        after = Epi::ahead(p, next, next.m * 256 + row_in, half);
      }
      if (x.k0 == x.k1) {
        if (t + clusters < total) Epi::more(p, next, next.m * 256 + row_in, half, after);
        continue;
      }
      const uint32_t buf = tile & 1;
      if (!__all_sync(0xffffffffu, tc_wait(tc_smem(&sh.acc_full[buf]), (tile >> 1) & 1, &sh, p.status, 4))) break;
      tc_fence_after();
      Epi::run(p, x, x.m * 256 + row_in, half, tmem + buf * 256 + ((uint32_t)(quad * 32) << 16),
               raw + (stages - tc_smem(raw)) + kTcRingBytes + (warp - 4) * kTcStoreBytes, state);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) tc_bar_arrive_remote(tc_smem(&sh.acc_empty[buf]), 0);
      ++tile;
      if (t + clusters < total) Epi::more(p, next, next.m * 256 + row_in, half, after);
    }
  }

  // teardown
  if (warp == 3 && lane == 0 && sh.give_up) {
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

// Launch on every SM pair that can hold a cluster, or fewer when there are
// fewer tiles or an SM budget.
template <bool AMN, bool BMN, class Epi>
cudaError_t tc_launch(const TcArgs& p, cudaStream_t s, int* grid_out) {
  constexpr auto kern = tc_gemm_kernel<AMN, BMN, Epi>;
  const cudaError_t attr = raise_smem<kern>(kTcSmem);
  if (attr != cudaSuccess) return attr;
  const int grid = 2 * tc_clusters(tc_units(p));
  if (grid_out) *grid_out = grid;
  return launch_pdl(kern, grid, kTcThreads, kTcSmem, s, p);
}

}  // namespace rra
