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
//
// An entry of dl is off by up to half a bfloat16 step, which averages out over
// the many small entries of a row but not for the target's, which alone is as
// large as all others together: a token's share of the gradients would be off
// by up to 2^-8 as a whole.  So the rest of the target's entry that bfloat16
// leaves, lo[t], is kept in float32 and added back where the products'
// epilogues still hold float32: lo[t] W[target] to row t of dx, lo[t] x[t] to
// row target of dW (dW of 333 x 515 x 50021 off by 0.0017 in the 2-norm
// against 0.0023 without).  Up to 32 tokens dW sums so few entries that their
// roundings do not average out either, and what bfloat16 leaves of every entry
// is stored too, as 32 rows more at most: a second K segment of dW's product (a
// shard's dW of 1 or 4 tokens x 346 off by 0.0017 against 0.0023-0.0025
// without; of 1 / 4 tokens x 5120 x 32768 253 / 243 us).
//
// Bound by the tensor cores: the epilogue's exponentials (one per logit, 4 a
// cycle and scheduler) run under the products of the next tile, and show for
// short rows only (2048 x 131072 of hidden 128 131 us).  Measured: forward 2048
// x 5120 x 131072 1.56-1.61 ms call after call (1.71-1.76 PFLOP/s, tensor pipe
// 96% active; 1.36 ms from a cool start); forward and backward of 8192 x 5120 x
// 131072 25.5-26.7 ms (1.65-1.72 PFLOP/s under the power limit, where a library
// product sustains 1.70).
#include "tc_epilogue.cuh"

namespace rra {

constexpr float kLog2e = 1.4426950408889634f;

// Thread `i` of `n`'s share of the dot product of two rows, in float32.
__device__ __forceinline__ float row_dot(const __nv_bfloat16* x, const __nv_bfloat16* w, long long hidden, int vec, int i,
                                         int n) {
  float dot = 0.f;
  if (vec) {
    for (long long c = i * 8; c < hidden; c += n * 8) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + c)), v = __ldg(reinterpret_cast<const uint4*>(w + c));
      const uint32_t p[4] = {u.x, u.y, u.z, u.w}, q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dot = fmaf(__uint_as_float(p[j] << 16), __uint_as_float(q[j] << 16), dot);
        dot = fmaf(__uint_as_float(p[j] & 0xFFFF0000u), __uint_as_float(q[j] & 0xFFFF0000u), dot);
      }
    }
  } else {
    for (long long c = i; c < hidden; c += n) dot = fmaf(__bfloat162float(x[c]), __bfloat162float(w[c]), dot);
  }
  return dot;
}

struct EpiLse : TcNoState {
  // (a - m) log2(e) and (b - m) log2(e), two to an instruction.
  static __device__ __forceinline__ void less_log2(float& a, float& b, float m) {
    asm("{\n.reg .b64 v, m, k;\n"
        "mov.b64 v, {%0, %1};\nmov.b64 m, {%2, %2};\nmov.b64 k, {%3, %3};\n"
        "sub.rn.f32x2 v, v, m;\nmul.rn.f32x2 v, v, k;\nmov.b64 {%0, %1}, v;\n}\n"
        : "+f"(a), "+f"(b)
        : "f"(m), "f"(kLog2e));
  }

  // One row's 32 logits into its running maximum and sum.  The maximum is
  // taken off before the change to base 2: its own exponential is 1 exactly
  // and a maximum that stays leaves the sum as it is, whatever its size (one
  // fused multiply-add of v log2(e) and the rounded m log2(e) would multiply
  // the sum by 2^d per 32 columns, d half a unit in the last place of the
  // latter: lse off by 1e-5 at logits of 100, 1e-4 at 1000).
  static __device__ __forceinline__ void chunk(const TcArgs& p, float* v, int valid, long long d, int row, float& m,
                                               float& s) {
    if (valid < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j >= valid) v[j] = -INFINITY;
    }
    if (d >= 0 && d < 32 && d < valid) {
      float h = v[0];  // a select per column: an indexed read would put v in local memory
#pragma unroll
      for (int j = 1; j < 32; ++j)
        asm("{\n.reg .pred p;\nsetp.eq.s32 p, %1, %2;\n@p mov.f32 %0, %3;\n}\n" : "+f"(h) : "r"((int)d), "r"(j), "f"(v[j]));
      p.hit[row] = h;
    }
    float q[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int j = 4; j < 32; ++j) q[j & 3] = fmaxf(q[j & 3], v[j]);
    const float nm = fmaxf(m, fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3])));
    if (nm == -INFINITY) {  // nothing but -inf so far (or NaN, which the maximum skips)
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (v[j] != v[j]) s = v[j];
    } else {
      float e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float a = v[j], b = v[j + 1];
        less_log2(a, b, nm);
        e[j & 3] += tc_exp2(a);
        e[(j & 3) + 1] += tc_exp2(b);
      }
      s = s * tc_exp2((m - nm) * kLog2e) + ((e[0] + e[1]) + (e[2] + e[3]));
      m = nm;
    }
  }

  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row0, int half, uint32_t addr,
                                             uint8_t*, const State&) {
    const TcGroup& g = p.group[x.group];
    const int row = row0 + (threadIdx.x & 31);
    const int c0 = x.n * 256 + half * 128;
    float m = -INFINITY, s = 0.f;
    long long t = -1;
    if (row < g.M) {
      t = p.targets[row];
      t = t == p.ignore_index ? -1 : t - (g.col0 + c0);
    }
    const int valid = g.N - c0;
    if (valid > 0) {
      // the next 32 columns are read from tensor memory under the exponentials of these
      float v[2][32];
      tc_ld32(addr + half * 128, v[0]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tc_ld_ready(v[c & 1]);
        if (c < 3) tc_ld32(addr + half * 128 + 32 * (c + 1), v[(c + 1) & 1]);
        if (32 * c < valid) chunk(p, v[c & 1], valid - 32 * c, t - 32 * c, row, m, s);
      }
      __syncwarp();
    }
    if (row < g.M) p.part[(long long)((g.part0 + x.n) * 2 + half) * p.part_ld + row] = make_float2(m, s);
  }
};

// REST: what bfloat16 leaves of each entry is stored too, p.rest_row rows on.
// A variant of its own: one kernel for both took 127 registers for 95 and 25.4
// to 25.6 ms for 25.0 to 25.1 (8192 x 5120 x 131072, both passes).
template <bool REST>
struct EpiDlogits : TcNoState {
  static __device__ __forceinline__ void run(const TcArgs& p, const TcTile& x, int row0, int half, uint32_t addr,
                                             uint8_t* buf, const State&) {
    const TcGroup& g = p.group[x.group];
    const int row = row0 + (threadIdx.x & 31);
    const int c0 = x.n * 256 + half * 128;
    long long t = -1;
    float4 q = make_float4(INFINITY, 0.f, 0.f, 0.f);
    if (row < g.M) {
      q = p.rows[row];
      t = q.z != 0.f ? p.targets[row] - (g.col0 + c0) : -1;
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(g.out) + (long long)row0 * g.ld + c0;
#pragma unroll 1
    for (int c = 0; c < 128; c += 64) {
      const int valid = g.N - c0 - c;
      if (valid <= 0) break;
      uint32_t rest[REST ? 32 : 1];
#pragma unroll(REST ? 2 : 1)
      for (int k = 0; k < 64; k += 32) {
        float v[32];
        tc_ld32(addr + half * 128 + c + k, v);
        tc_ld_ready(v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = tc_exp2(fmaf(v[j], kLog2e, -q.x)) * q.w;
        const long long d = t - c - k;
        if (d >= 0 && d < 32) {  // the target's column, in one chunk of a row
#pragma unroll
          for (int j = 0; j < 32; ++j)
            asm("{\n.reg .pred p;\nsetp.eq.s32 p, %1, %2;\n@p mov.f32 %0, %3;\n}\n" : "+f"(v[j]) : "r"((int)d), "r"(j), "f"(q.y));
        }
        if (q.z == 0.f) {  // a row with no gradient, whatever its logits
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
        tc_stage_bf16(buf, v, k / 8);
        if (REST) tc_left2(v, rest + k / 2);
      }
      tc_flush_bf16(buf, out + c, g.ld, g.M - row0, valid, true, true);
      if (REST) {
        tc_stage_packed(buf, rest, 0);
        tc_stage_packed(buf, rest + 16, 4);
        tc_flush_bf16(buf, out + c + p.rest_row * g.ld, g.ld, g.M - row0, valid, true, true);
      }
    }
  }
};

cudaError_t launch_tc_lse(const TcArgs& p, cudaStream_t s, int* grid) {
  return tc_launch<false, false, EpiLse>(p, s, grid);
}

cudaError_t launch_tc_dlogits(const TcArgs& p, cudaStream_t s, int* grid) {
  return p.rest_row ? tc_launch<false, false, EpiDlogits<true>>(p, s, grid)
                    : tc_launch<false, false, EpiDlogits<false>>(p, s, grid);
}

// What the backward pass needs beside the logits.  The first row_ctas CTAs
// take the tokens, the CTAs from index0 on the index (under an SM budget all of
// them both), per token: {lse in units of log 2, the target's entry in
// bfloat16, 1 if the row has a gradient, grad}, the target (-1: none) and
// what bfloat16 leaves of its entry.  The index of the tokens by target: a warp per token counts the tokens that come before it, a warp
// per block of 32 vocabulary rows those before the block: tokens x (tokens +
// V / 32) comparisons (0.06 ms for 8192 tokens and 131072 rows), and no order
// that depends on timing.
struct RowsArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w[kMaxRanks];
  long long first[kMaxRanks + 1];
  int block0[kMaxRanks + 1];  // blocks of 32 rows of the shards before
  const long long* targets;
  long long ignore_index;
  const float* lse;
  const float* grad;
  float4* rows;
  int* column;
  float* lo;
  int* start;
  int* token;
  int* sorted;
  int hidden, nranks, vec, tokens, row_ctas, index0, items;
};

__device__ __forceinline__ long long live_target(const RowsArgs& a, int row) {
  const long long t = __ldg(a.targets + row);
  return t != a.ignore_index && t >= 0 && t < a.first[a.nranks] ? t : -1;
}

// A warp takes kIndexItems items at a time, so that each target it reads is
// compared with all of them.
constexpr int kIndexItems = 8;

__device__ __forceinline__ void loss_index(const RowsArgs& a) {
  const int lane = threadIdx.x & 31, ctas = gridDim.x - a.index0;
  for (int i0 = ((blockIdx.x - a.index0) * 8 + (threadIdx.x >> 5)) * kIndexItems; i0 < a.items;
       i0 += ctas * 8 * kIndexItems) {
    int key[kIndexItems];  // targets before this one count (-1: nothing to place)
    int tie[kIndexItems];  // and equal ones of tokens before this one
    int n[kIndexItems];
#pragma unroll
    for (int j = 0; j < kIndexItems; ++j) {
      const int i = i0 + j;
      key[j] = -1;
      tie[j] = n[j] = 0;
      if (i < a.tokens) {
        key[j] = (int)live_target(a, i);
        tie[j] = i;
      } else if (i < a.items) {
        const int b = i - a.tokens;
        int r = 0;
        while (r < a.nranks && b >= a.block0[r + 1]) ++r;
        key[j] = (int)(r == a.nranks ? a.first[a.nranks] : a.first[r] + 32ll * (b - a.block0[r]));
      }
    }
#pragma unroll 4
    for (int t = lane; t < a.tokens; t += 32) {
      const int live = (int)live_target(a, t), c = live < 0 ? 0x7FFFFFFF : live;
#pragma unroll
      for (int j = 0; j < kIndexItems; ++j) n[j] += c < key[j] + (t < tie[j] ? 1 : 0);
    }
#pragma unroll
    for (int j = 0; j < kIndexItems; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n[j] += __shfl_xor_sync(0xffffffffu, n[j], o);
      const int i = i0 + j;
      if (lane == 0 && key[j] >= 0) {
        if (i < a.tokens) {
          a.token[n[j]] = i;
          a.sorted[n[j]] = key[j];
        } else {
          a.start[i - a.tokens] = n[j];
        }
      }
    }
  }
}

// R rows at a time per CTA: 256 / R threads a row.
template <int R>
__device__ __forceinline__ void loss_row(const RowsArgs& a, int block, float* part) {
  constexpr int PER = 256 / R;
  const int row = block * R + threadIdx.x / PER, i = threadIdx.x % PER;
  const long long t = row < a.tokens ? live_target(a, row) : -1;
  float l = 0.f;
  if (t >= 0) {
    int g = 0;
    while (t >= a.first[g + 1]) ++g;
    l = row_dot(a.x + (long long)row * a.hidden, a.w[g] + (t - a.first[g]) * a.hidden, a.hidden, a.vec, i, PER);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (R == 1) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = l;
    __syncthreads();
    l = part[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) l += part[w];
  }
  if (i != 0 || row >= a.tokens) return;
  float4 q = make_float4(INFINITY, 0.f, 0.f, 0.f);
  float rest = 0.f;
  if (t >= 0) {
    const float lse = a.lse[row], grad = a.grad[row];
    const float d = l - lse;
    const float entry = (d < 0.f ? expm1f(d) : d != d ? d : 0.f) * grad;  // (p - 1) grad
    const float held = __bfloat162float(__float2bfloat16_rn(entry));
    q = make_float4(lse * kLog2e, held, 1.f, grad);
    rest = fabsf(held) < INFINITY ? entry - held : 0.f;
  }
  a.rows[row] = q;
  a.column[row] = (int)t;
  a.lo[row] = rest;
}

template <int R>
__global__ void __launch_bounds__(256) loss_rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float part[8];
  pdl_wait();
  pdl_next();
  if ((int)blockIdx.x < a.row_ctas) {
    for (int b = blockIdx.x; b * R < a.tokens; b += a.row_ctas) {
      loss_row<R>(a, b, part);
      if (R == 1) __syncthreads();  // part is free
    }
  }
  if ((int)blockIdx.x >= a.index0) loss_index(a);
}

cudaError_t launch_loss_rows(const void* x, const void* const* w, const size_t* vocab, int n, size_t hidden, int tokens,
                             const long long* targets, long long ignore_index, const float* lse, const float* grad,
                             float4* rows, int* column, float* lo, int* start, int* token, int* sorted,
                             cudaStream_t s) {
  RowsArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  for (int r = 0; r < n; ++r) {
    a.w[r] = static_cast<const __nv_bfloat16*>(w[r]);
    a.first[r + 1] = a.first[r] + (long long)vocab[r];
    a.block0[r + 1] = a.block0[r] + (int)((vocab[r] + 31) / 32);
  }
  a.targets = targets;
  a.ignore_index = ignore_index;
  a.lse = lse;
  a.grad = grad;
  a.rows = rows;
  a.column = column;
  a.lo = lo;
  a.start = start;
  a.token = token;
  a.sorted = sorted;
  a.hidden = (int)hidden;
  a.nranks = n;
  a.vec = hidden % 8 == 0;  // the matrices themselves are 16-byte aligned
  a.tokens = tokens;
  a.items = tokens + a.block0[n] + 1;
  const int per = 8 * kIndexItems, most = device_sms() * 8, want = (a.items + per - 1) / per;
  const int index_ctas = want < most ? want : most;
  // one row per CTA while that leaves SMs idle, else 8
  const bool few = tokens < 8 * device_sms();
  a.row_ctas = a.index0 = few ? tokens : (tokens + 7) / 8;
  const int grid = budget((size_t)a.row_ctas + index_ctas);
  if (grid < a.row_ctas + index_ctas) {
    a.row_ctas = grid;
    a.index0 = 0;
  }
  return few ? launch_pdl(loss_rows_kernel<1>, grid, 256, 0, s, a)
             : launch_pdl(loss_rows_kernel<8>, grid, 256, 0, s, a);
}

// Join the column parts of each row, R rows per CTA at a time (256 threads: 256 / R
// threads a row, lanes of neighbouring rows side by side so that loads of
// the [part][row] array stay whole sectors), and refine the target's logit.
//
// The tensor cores truncate each partial sum of a product: 320 of them at
// hidden 5120 leave a logit about 2e-6 low relative to its terms, and the
// loss carries that of the target's logit in full.  So the target's logit l
// is computed once more as a plain float32 sum, and takes the place of the
// product's value l' both in the loss and inside lse:
//   d = l - l',  c = log(1 + exp(l' - lse')(exp(d) - 1))
//   lse = lse' + c,  loss = (lse' - l') - d + c
// which stays accurate when the target carries nearly all of the mass, where
// lse' - l alone would lose d.  lse' stays in two parts until then, the
// maximum m and log s, which rounding their sum would cut to the steps of m.
struct JoinArgs {
  const float2* part;
  long long part_ld;
  int parts, rows, nranks;
  const float* hit;
  const long long* targets;
  long long ignore_index;
  const __nv_bfloat16* x;
  const __nv_bfloat16* w[kMaxRanks];
  long long first[kMaxRanks + 1];  // the shards' first columns
  long long hidden;
  int vec;  // rows of x and w start on 16 bytes
  float* loss;
  float* lse;
};

__device__ __forceinline__ void join_one(float& m, float& s, float2 q) {
  const float nm = fmaxf(m, q.x);
  if (nm == -INFINITY) {
    s += q.y;  // 0, or NaN
  } else {
    s = s * expf(m - nm) + q.y * expf(q.x - nm);
    m = nm;
  }
}

template <int R>
__device__ __forceinline__ void join_rows(const JoinArgs& a, int row0, float2* red, float* dots) {
  constexpr int PER = 256 / R;  // threads a row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = tid % R, k = tid / R;
  const int row = row0 + r;
  float m = -INFINITY, s = 0.f;
  if (row < a.rows) {
    const float2* p = a.part + row;
    int i = k;
    for (; i + 3 * PER < a.parts; i += 4 * PER) {
      float2 q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = __ldg(p + (long long)(i + j * PER) * a.part_ld);
#pragma unroll
      for (int j = 0; j < 4; ++j) join_one(m, s, q[j]);
    }
    for (; i < a.parts; i += PER) join_one(m, s, __ldg(p + (long long)i * a.part_ld));
  }
  red[tid] = make_float2(m, s);

  // the target's logit in float32: a warp per row (R = 8), or all for the one
  const int drow = R == 1 ? row0 : row0 + warp;
  const int dt = R == 1 ? tid : lane, dn = R == 1 ? 256 : 32;
  float dot = 0.f;
  bool inside = false;
  if (drow < a.rows) {
    const long long t = a.targets[drow];
    inside = t != a.ignore_index && t >= 0 && t < a.first[a.nranks];
    if (inside) {
      int g = 0;
      while (t >= a.first[g + 1]) ++g;
      const __nv_bfloat16* w = a.w[g] + (t - a.first[g]) * a.hidden;
      const __nv_bfloat16* x = a.x + (long long)drow * a.hidden;
      dot = row_dot(x, w, a.hidden, a.vec, dt, dn);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (lane == 0) dots[warp] = dot;
#pragma unroll
  for (int half = PER / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (k < half) {
      join_one(m, s, red[tid + half * R]);
      red[tid] = make_float2(m, s);
    }
  }
  __syncthreads();
  if (k == 0 && row < a.rows) {
    const float rest = logf(s);  // NaN as s
    float l = s != s ? s : m + rest;
    const long long t = a.targets[row];
    float out = 0.f;
    if (t != a.ignore_index) {
      if (t < 0 || t >= a.first[a.nranks]) {
        out = NAN;
      } else {
        float fine = dots[R == 1 ? 0 : r];
        if (R == 1)
          for (int i = 1; i < 8; ++i) fine += dots[i];
        const float rough = a.hit[row];
        const float d = fabsf(fine) < INFINITY && fabsf(rough) < INFINITY ? fine - rough : 0.f;
        const float top = m - rough;  // what the maximum is above the product's logit
        const float c = d != 0.f ? log1pf(expf(-top - rest) * expm1f(d)) : 0.f;
        out = (top - d) + (rest + c);
        l = m + (rest + c);
      }
    }
    a.lse[row] = l;
    a.loss[row] = out;
  }
}

// LOOP: every gridDim-th R rows (an SM budget leaves fewer CTAs).
template <int R, bool LOOP>
__global__ void __launch_bounds__(256) loss_join_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ float2 red[256];
  __shared__ float dots[8];
  pdl_wait();
  pdl_next();
  int row0 = blockIdx.x * R;
  do {
    join_rows<R>(a, row0, red, dots);
    row0 += gridDim.x * R;
    if (LOOP) __syncthreads();  // red and dots are free
  } while (LOOP && row0 < a.rows);
}

template <int R>
static cudaError_t join_go(const JoinArgs& a, cudaStream_t s) {
  const int want = (a.rows + R - 1) / R, grid = budget(want);
  return launch_pdl(grid < want ? loss_join_kernel<R, true> : loss_join_kernel<R, false>, grid, 256, 0, s, a);
}

cudaError_t launch_loss_join(const float2* part, int parts, const float* hit, const long long* targets,
                             long long ignore_index, const void* x, const void* const* w, const size_t* vocab, int n,
                             size_t hidden, int rows, float* loss, float* lse, cudaStream_t s) {
  JoinArgs a{};
  a.part = part;
  a.part_ld = rows;
  a.parts = parts;
  a.rows = rows;
  a.nranks = n;
  a.hit = hit;
  a.targets = targets;
  a.ignore_index = ignore_index;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.hidden = (long long)hidden;
  a.vec = hidden % 8 == 0;  // the matrices themselves are 16-byte aligned
  for (int r = 0; r < n; ++r) {
    a.w[r] = static_cast<const __nv_bfloat16*>(w[r]);
    a.first[r + 1] = a.first[r] + (long long)vocab[r];
  }
  a.loss = loss;
  a.lse = lse;
  // one row per CTA while that leaves SMs idle, else 8 (whole sectors of parts)
  return rows < 8 * device_sms() ? join_go<1>(a, s) : join_go<8>(a, s);
}

}  // namespace rra
