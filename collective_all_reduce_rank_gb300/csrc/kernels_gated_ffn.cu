// kernels_gated_ffn.cu -- the column-parallel half of a gated feed-forward
// block over the virtual ranks' weight shards:
//
//   g_r = x G_r^T,  u_r = x U_r^T,  a_r = act(g_r) * u_r
//
// Both projections, the activation and the product run in one kernel: a
// tile's 256 accumulator columns are 128 gate columns and the same 128 up
// columns (the first CTA of a pair stages gate rows, the second up rows), so
// a thread finds g and u of one element in its own tensor-memory lane.  The
// backward pass computes g and u again the same way and its epilogue turns
// them and da into dg = da u act'(g) and du = da act(g), rounded to
// bfloat16 (operands of the two gradient products, kernels_tc_store.cu).
//
// That rounding makes both gradients 1.41 times as far from their exact values
// as their own rounding does (0.0024 against 0.0017 in the 2-norm), where many
// entries take part; where one token's few entries carry a shard's gradient,
// up to 2.1 times (one to 18 tokens).  Up to 128 tokens what bfloat16 leaves of
// each entry is stored too, as rows behind the tokens': more rows of the same
// tile for dx, added in the join, and a second K segment for dG and dU.  Both
// are then off by their own rounding alone, for 1 to 13 us: 1 / 32 / 64 / 128
// tokens x 5120 x 8 x 1728 219 / 224 / 233 / 243 us (213 / 217 / 223 / 230
// without), 32 x 1027 x 3 x 643 44 (41), 128 x 512 x 4 x 512 32 (28).
//
// Bound by the tensor cores from about 300 tokens (512 x 5120 x 8 x 1728: 97-
// 100 us call after call, 1.45-1.50 PFLOP/s, and 85 us in a graph from a cool
// start; 224 tiles on 76 clusters are 2.95 waves), by the
// weights' bytes below (17-256 tokens: 56-61 us, 5.0-4.6 TB/s: 112 tiles are
// 1.5 waves and each tile's products take as long as its bytes); up to 16
// tokens go through kernels_skinny.cu.  Tiles of 64 + 64 columns fill the
// waves better but measured slower (65 us).
#include "act.cuh"
#include "tc_epilogue.cuh"

namespace rra {

template <int ACT>
struct EpiGate : TcNoState {
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row0, int half, uint32_t addr,
                                             uint8_t* buf, const State&) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 128 + half * 64;
    const int valid = g.N - c0;
    if (valid <= 0) return;
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
      float a[32], b[32];
      tc_ld32(addr + half * 64 + c, a);
      tc_ld32(addr + 128 + half * 64 + c, b);
      tc_ld_ready(a);
      tc_ld_ready(b);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float unused;
        a[j] = a[j] * gate_sigma<ACT>(a[j], &unused) * b[j];
      }
      tc_stage_bf16(buf, a, c / 8);
    }
    tc_flush_bf16(buf, static_cast<__nv_bfloat16*>(g.out) + (long long)row0 * g.ld + c0, g.ld, g.M - row0, valid,
                  g.vec, false);
  }
};

// REST: what bfloat16 leaves of each entry is stored too, p.rest_row rows on.
template <int ACT, bool REST>
struct EpiGateBack : TcNoState {
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row0, int half, uint32_t addr,
                                             uint8_t* buf, const State&) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 128 + half * 64;
    const int rows = g.M - row0;
    if (rows <= 0) return;  // few tokens: most warps have none
    const long long off = (long long)row0 * g.ld + c0;
    const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(g.in) + (long long)row0 * g.ld_in + c0;
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
      const int valid = g.N - c0 - c;
      if (valid <= 0) break;
      float a[32], b[32], d[32];
      tc_ld32(addr + half * 64 + c, a);
      tc_ld32(addr + 128 + half * 64 + c, b);
      tc_load_bf16(buf, in + c, g.ld_in, rows, valid, g.vec, d);
      tc_ld_ready(a);
      tc_ld_ready(b);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float k;
        const float s = gate_sigma<ACT>(a[j], &k);
        const float h = a[j] * s;  // act(g)
        const float slope = gate_slope<ACT>(a[j], s, k);
        a[j] = d[j] * b[j] * slope;
        b[j] = d[j] * h;
      }
      // 32 columns of dg in the first half of the staged rows, of du in the second
      __nv_bfloat16 *dg = static_cast<__nv_bfloat16*>(g.out) + off + c, *du = static_cast<__nv_bfloat16*>(g.out2) + off + c;
      tc_stage_bf16(buf, a, 0);
      tc_stage_bf16(buf, b, 4);
      uint32_t la[REST ? 16 : 1], lb[REST ? 16 : 1];
      if (REST) {
        tc_left2(a, la);
        tc_left2(b, lb);
      }
      tc_flush_pair(buf, dg, du, g.ld, rows, valid);
      if (REST) {
        tc_stage_packed(buf, la, 0);
        tc_stage_packed(buf, lb, 4);
        tc_flush_pair(buf, dg + p.rest_row * g.ld, du + p.rest_row * g.ld, g.ld, rows, valid);
      }
    }
  }
};

cudaError_t launch_tc_gate(const TcArgs& p, cudaStream_t s, int* grid) {
  return p.act == RRA_ACT_SILU ? tc_launch<false, false, EpiGate<RRA_ACT_SILU>>(p, s, grid)
                               : tc_launch<false, false, EpiGate<RRA_ACT_GELU_TANH>>(p, s, grid);
}

cudaError_t launch_tc_gate_back(const TcArgs& p, cudaStream_t s, int* grid) {
  if (p.rest_row)
    return p.act == RRA_ACT_SILU ? tc_launch<false, false, EpiGateBack<RRA_ACT_SILU, true>>(p, s, grid)
                                 : tc_launch<false, false, EpiGateBack<RRA_ACT_GELU_TANH, true>>(p, s, grid);
  return p.act == RRA_ACT_SILU ? tc_launch<false, false, EpiGateBack<RRA_ACT_SILU, false>>(p, s, grid)
                               : tc_launch<false, false, EpiGateBack<RRA_ACT_GELU_TANH, false>>(p, s, grid);
}

}  // namespace rra
