// kernels_vocab_loss.cu -- softmax cross entropy over a vocabulary held as
// shards of the virtual ranks, without keeping the logits.
//
//   l[t][v] = x[t] . W[v],  lse[t] = log sum_v exp l[t][v],
//   loss[t] = lse[t] - l[t][target[t]]
//   dl[t][v] = (exp(l[t][v] - lse[t]) - [v == target[t]]) grad[t]
//
// Forward: the product's epilogue reduces each row of a 256 x 256 tile of
// logits in registers to a running maximum and sum per 128 columns, and the
// thread that meets the target's column stores that logit; a second kernel
// joins the parts.  Backward, in pieces of the vocabulary: the logits are
// computed again and the epilogue stores dl of the piece in bfloat16, from
// which the two gradient products (kernels_tc_store.cu) read it.
#include "tc_epilogue.cuh"

namespace rra {

constexpr float kLog2e = 1.4426950408889634f;

struct EpiLse {
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row, int half, uint32_t addr) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 256 + half * 128;
    float m = -INFINITY, s = 0.f;
    long long t = -1;
    if (row < g.M) {
      t = p.targets[row];
      t = t == p.ignore_index ? -1 : t - (g.col0 + c0);
    }
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      const int valid = g.N - c0 - c;
      if (valid <= 0) break;
      float v[32];
      tc_ld32(addr + half * 128 + c, v);
      tc_ld_wait();
      if (valid < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j >= valid) v[j] = -INFINITY;
      }
      const long long d = t - c;
      if (d >= 0 && d < 32 && d < valid) {
        float h = v[0];
#pragma unroll
        for (int j = 1; j < 32; ++j)
          if (j == (int)d) h = v[j];
        p.hit[row] = h;
      }
      float q = v[0];
#pragma unroll
      for (int j = 1; j < 32; ++j) q = fmaxf(q, v[j]);
      const float nm = fmaxf(m, q);
      if (nm == -INFINITY) {  // nothing but -inf so far (or NaN, which the maximum skips)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (v[j] != v[j]) s = v[j];
        continue;
      }
      const float base = nm * kLog2e;
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        a += exp2f(fmaf(v[j], kLog2e, -base));
        b += exp2f(fmaf(v[j + 1], kLog2e, -base));
      }
      s = s * exp2f(fmaf(m, kLog2e, -base)) + (a + b);
      m = nm;
    }
    if (row < g.M) p.part[(long long)((g.part0 + x.n) * 2 + half) * p.part_ld + row] = make_float2(m, s);
  }
};

struct EpiDlogits {
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row, int half, uint32_t addr) {
    const TcGroup& g = p.group[x.group];
    const int c0 = x.n * 256 + half * 128;
    long long t = -1;
    float base = 0.f, w = 0.f;
    bool live = false;
    if (row < g.M) {
      const long long tgt = p.targets[row];
      // an ignored row, or one whose target lies outside the vocabulary, has a zero gradient
      live = tgt != p.ignore_index && tgt >= 0 && tgt < p.vocab;
      t = live ? tgt - (g.col0 + c0) : -1;
      base = p.lse[row] * kLog2e;
      w = p.grad[row];
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(g.out) + (long long)row * g.ld + c0;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      const int valid = g.N - c0 - c;
      if (valid <= 0) break;
      float v[32];
      tc_ld32(addr + half * 128 + c, v);
      tc_ld_wait();
      if (row >= g.M) continue;
      const int d = t - c >= 0 && t - c < 32 ? (int)(t - c) : -1;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float e = exp2f(fmaf(v[j], kLog2e, -base)) - (j == d ? 1.f : 0.f);
        v[j] = live ? e * w : 0.f;
      }
      tc_store_bf16(out + c, v, valid, true, true);
    }
  }
};

cudaError_t launch_tc_lse(const TcArgs& p, cudaStream_t s, int* grid) {
  return tc_launch<false, false, EpiLse>(p, s, grid);
}

cudaError_t launch_tc_dlogits(const TcArgs& p, cudaStream_t s, int* grid) {
  return tc_launch<false, false, EpiDlogits>(p, s, grid);
}

// Join the column parts of 32 rows per CTA: 8 threads a row, each over every
// 8th part, then across the 8 through shared memory, in a fixed order.
__global__ void __launch_bounds__(256)
    loss_join_kernel(const float2* part, long long part_ld, int parts, const float* hit, const long long* targets,
                     long long ignore_index, long long vocab, int rows, float* loss, float* lse) {
  __shared__ float2 red[8][32];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.f;
  if (row < rows) {
    for (int i = k; i < parts; i += 8) {
      const float2 q = __ldg(part + (long long)i * part_ld + row);
      const float nm = fmaxf(m, q.x);
      if (nm == -INFINITY) {
        s += q.y;  // 0, or NaN
      } else {
        s = s * expf(m - nm) + q.y * expf(q.x - nm);
        m = nm;
      }
    }
  }
  red[k][lane] = make_float2(m, s);
  __syncthreads();
  if (k == 0 && row < rows) {
    for (int i = 1; i < 8; ++i) {
      const float2 q = red[i][lane];
      const float nm = fmaxf(m, q.x);
      if (nm == -INFINITY) {
        s += q.y;
      } else {
        s = s * expf(m - nm) + q.y * expf(q.x - nm);
        m = nm;
      }
    }
    const float l = s != s ? s : m + logf(s);
    lse[row] = l;
    const long long t = targets[row];
    if (loss) loss[row] = t == ignore_index ? 0.f : (t < 0 || t >= vocab ? NAN : l - hit[row]);
  }
}

cudaError_t launch_loss_join(const float2* part, long long part_ld, int parts, const float* hit,
                             const long long* targets, long long ignore_index, long long vocab, int rows,
                             float* loss, float* lse, cudaStream_t s) {
  loss_join_kernel<<<(rows + 31) / 32, 256, 0, s>>>(part, part_ld, parts, hit, targets, ignore_index, vocab, rows,
                                                    loss, lse);
  return cudaGetLastError();
}

}  // namespace rra
