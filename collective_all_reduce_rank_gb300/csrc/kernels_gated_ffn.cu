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
// Bound by the tensor cores from about 300 tokens (512 x 5120 x 8 x 1728: 84
// us, 1.73 PFLOP/s; 224 tiles on 76 clusters are 2.95 waves), by the
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

template <int ACT>
struct EpiGateBack : TcNoState {
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row0, int half, uint32_t addr,
                                             uint8_t* buf, const State&) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 128 + half * 64;
    const int rows = g.M - row0;
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
      tc_stage_bf16(buf, a, 0);
      tc_stage_bf16(buf, b, 4);
      tc_flush_pair(buf, static_cast<__nv_bfloat16*>(g.out) + off + c, static_cast<__nv_bfloat16*>(g.out2) + off + c,
                    g.ld, rows, valid);
    }
  }
};

cudaError_t launch_tc_gate(const TcArgs& p, cudaStream_t s, int* grid) {
  return p.act == RRA_ACT_SILU ? tc_launch<false, false, EpiGate<RRA_ACT_SILU>>(p, s, grid)
                               : tc_launch<false, false, EpiGate<RRA_ACT_GELU_TANH>>(p, s, grid);
}

cudaError_t launch_tc_gate_back(const TcArgs& p, cudaStream_t s, int* grid) {
  return p.act == RRA_ACT_SILU ? tc_launch<false, false, EpiGateBack<RRA_ACT_SILU>>(p, s, grid)
                               : tc_launch<false, false, EpiGateBack<RRA_ACT_GELU_TANH>>(p, s, grid);
}

}  // namespace rra
