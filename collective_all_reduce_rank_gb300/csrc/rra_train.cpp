// rra_train.cpp -- the C ABI of the training-step operators: argument
// checks, workspace plans, tensor maps and the sequence of launches.  All
// computation runs in kernels_norm8.cu, kernels_gated_ffn.cu,
// kernels_vocab_loss.cu and kernels_tc_store.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <initializer_list>

#include "abi_util.h"
#include "rra.h"
#include "rra_internal.h"
#include "serve_host.h"
#include "tc_host.h"

using namespace rra;

namespace {

constexpr size_t kPieceBytes = 512ull << 20;  // default room for a piece's dl

size_t tiles256(size_t x) { return (x + 255) / 256; }

// A matrix a product reads: the caller's rows, or padded rows in the
// workspace.
struct Mat {
  const void* p;
  size_t rows, cols, ld;
};

// Bump allocation in the workspace; with a null base it only counts.
struct Bump {
  char* base;
  size_t at = 0;
  void* take(size_t bytes) {
    void* p = base ? base + at : nullptr;
    at += up(bytes, kAlign);
    return p;
  }
};

size_t slot_ld(size_t hidden) { return up(hidden, 8); }  // float32 rows of dx's parts
bool padded(size_t hidden) { return hidden % 8 != 0; }
size_t pad_ld(size_t hidden) { return up(hidden, 64); }  // rows of whole 128-byte lines

// The rows products read of the caller's matrices: copied to padded rows
// when needed, all of them in one launch.
struct Placer {
  Bump& ws;
  PadArgs a{};
  explicit Placer(Bump& w) : ws(w) {}
  Mat operator()(const void* p, size_t rows, size_t cols) {
    Mat m{p, rows, cols, cols};
    if (!padded(cols)) return m;
    m.ld = pad_ld(cols);
    m.p = ws.take(rows * m.ld * 2);
    if (rows == 0) return m;
    a.src[a.n] = p;
    a.dst[a.n] = const_cast<void*>(m.p);
    a.cols = (long long)m.cols;
    a.units = (int)(m.ld / 8);
    a.first[a.n + 1] = a.first[a.n] + (long long)rows * a.units;
    ++a.n;
    return m;
  }
  bool launch(cudaStream_t s) { return a.n == 0 || launch_pad_rows(a, s) == cudaSuccess; }
};

bool map_k(CUtensorMap* m, const Mat& x, int box = 128) { return tc_map(m, x.p, x.cols, x.rows, x.ld, false, box); }
bool map_mn(CUtensorMap* m, const Mat& x) { return tc_map(m, x.p, x.cols, x.rows, x.ld, true, 64); }

void clear(TcArgs* p) { *p = TcArgs{}; }

// What a product of `tokens` rows of A stages.
TcShape pick_shape(size_t tokens) {
  TcShape q;
  if (tokens > 128) return q;
  q.a_rows = (int)up(tokens, 8);
  q.a_ctas = 1;
  q.stages = 6 * 32768 / (q.a_rows * 128 + 16384);  // 8 rows: 11, below kTcMaxStages
  return q;
}

// How an input gradient's tiles are spread over the clusters: `full` whole
// tiles in whole waves, and the rest split into `splits` parts of the K axis
// that run side by side, so that the last wave is as short as its share of
// the work (4096 x 5120: 320 tiles on 76 clusters are 4 waves and 16 tiles,
// which unsplit take a fifth: 0.72 against 0.64 ms).  The count minimises
// the waves of products (0.27 us for the 64-deep step of a tile, measured on
// the full kernel) plus the join: 5 us, and 0.05 us for each part's 256 KB
// written and read (777 tokens x 1027, 20 tiles of 66 steps: 28 us unsplit,
// 16 + 6 us in 3 parts).
struct Split {
  int full = 0, splits = 1;
  size_t slot_bytes = 0;
};

Split pick_split(size_t tokens, size_t hidden, size_t kblocks) {
  Split q;
  const long long tiles = (long long)(tiles256(tokens) * tiles256(hidden));
  const long long clusters = std::max(1, device_sms() / 2);
  const long long full = tiles / clusters * clusters, rest = tiles - full;
  double best = 1e30;
  for (int s = 1; s <= 64 && (size_t)s * 4 <= std::max<size_t>(kblocks, 4); ++s) {
    const double waves = (double)((rest * s + clusters - 1) / clusters) / s;
    const double us = waves * 0.27 * (double)kblocks + (s > 1 ? 5.0 + (double)(rest * s) * 0.05 : 0.0);
    if (us < best * 0.97) {
      best = us;
      q.splits = s;
    }
  }
  q.full = (int)(q.splits > 1 ? full : tiles);
  q.slot_bytes = q.splits > 1 ? (size_t)rest * q.splits * 65536 * 4 : 0;
  return q;
}

bool add_group(TcArgs* p, const TcGroup& g0, bool pair) {
  TcGroup g = g0;
  g.mt = (int)tiles256((size_t)g.M);
  g.nt = pair ? (g.N + 127) / 128 : (int)tiles256((size_t)g.N);
  const long long t = (long long)g.mt * g.nt + p->tiles;
  if (t > INT_MAX / 2 || p->ngroups >= kTcMaxGroups) return false;
  g.tile0 = p->tiles;
  p->group[p->ngroups++] = g;
  p->tiles = (int)t;
  return true;
}

void one_k_axis(TcArgs* p, size_t k) {
  p->nsegs = 1;
  p->seg_k0[0] = 0;
  p->kblocks = (int)((k + kTcKBlock - 1) / kTcKBlock);
  p->splits = 1;
  p->full = p->tiles;
}

// A K axis of T tokens, and with `rest` once more: B's rows again, against the
// rows of A behind the first T (what bfloat16 leaves of those).  A block that
// runs past T meets zeros of B.
void token_axis(TcArgs* p, size_t T, bool rest) {
  one_k_axis(p, T);
  if (!rest) return;
  p->rest_k = (int)T;
  p->nsegs = 2;
  p->seg_k0[1] = p->kblocks;
  p->kblocks *= 2;
}

// More 256 x 256 tiles than the walk can count (`extra`: shards, each of
// which may end in a partial tile).
bool too_many_tiles(size_t m, size_t n, size_t extra) {
  return (tiles256(m) + extra) * (tiles256(n) + extra) > (size_t)INT_MAX / 4;
}

bool bad_extent(size_t a) { return a > (size_t)INT_MAX - 1024; }

using Fn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                        const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                        CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Fn encode_fn() {
  static const Fn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (Fn) nullptr;
    return (Fn)p;
  }();
  return fn;
}

thread_local int g_largest_grid = 0;

}  // namespace

void rra::note_grid(int grid) { g_largest_grid = std::max(g_largest_grid, grid); }

int rra::take_grid() {
  const int g = g_largest_grid;
  g_largest_grid = 0;
  return g;
}

// ---------------------------------------------------------------------------
// shared with the kernels
// ---------------------------------------------------------------------------

bool rra::tc_map(CUtensorMap* m, const void* base, size_t inner, size_t rows, size_t ld, bool mn_major, int box_rows) {
  const Fn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rra::mx4_map_codes(CUtensorMap* m, const void* base, size_t row_bytes, size_t rows, int box_rows) {
  const Fn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rra::mx4_map_scales(CUtensorMap* m, const void* base, size_t across, size_t bands, int box_bands) {
  const Fn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {across * 128, bands};  // words
  const cuuint64_t strides[1] = {across * 512};
  const cuuint32_t box[2] = {256, (cuuint32_t)box_bands};
  const cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int rra::tc_clusters(int tiles) {
  int c = device_sms() / 2;
  if (max_ctas_cap() > 0) c = std::min(c, std::max(1, max_ctas_cap() / 2));
  return std::max(1, std::min(c, tiles));
}

// ---------------------------------------------------------------------------
// norm with an 8-bit checkpoint
// ---------------------------------------------------------------------------

namespace {

rra_status_t norm_common(const void* const* a, void* const* b, int n, size_t rows, size_t hidden, const void* gamma,
                         int dt) {
  if (!a || !b || !gamma || n < 1 || (dt != RRA_FLOAT32 && dt != RRA_BFLOAT16) || hidden == 0)
    return n > kMaxRanks ? RRA_ERR_UNSUPPORTED : RRA_ERR_INVALID_ARG;
  if (n > kMaxRanks || hidden > kNormMaxHidden || rows > 0x7FFFFFFFull) return RRA_ERR_UNSUPPORTED;
  const size_t e = dt == RRA_BFLOAT16 ? 2 : 4;
  if (rows && hidden > (SIZE_MAX / 4) / rows / e) return RRA_ERR_INVALID_ARG;
  if (!aligned(gamma, e)) return RRA_ERR_INVALID_ARG;
  for (int r = 0; r < n; ++r)
    if ((rows && (!a[r] || !b[r])) || !aligned(a[r], e) || !aligned(b[r], e)) return RRA_ERR_INVALID_ARG;
  return RRA_SUCCESS;
}

bool norm_vec(const void* const* a, const void* const* b, int n, const void* gamma, const void* codes, size_t hidden,
              size_t e) {
  bool v = aligned(gamma, 16) && aligned(codes, 16) && (hidden * e) % 16 == 0;
  for (int r = 0; r < n; ++r) v = v && (!a || aligned(a[r], 16)) && aligned(b[r], 16);
  return v;
}

}  // namespace

extern "C" {

rra_status_t rra_allreduce_rmsnorm_save8(const void* const* bufs, void* const* outs, int nranks, size_t rows,
                                         size_t hidden, const void* gamma, float eps, void* codes, void* scales,
                                         float* rstd, rra_dtype_t dtype, rra_stream_t stream) {
  const char* call = "allreduce_rmsnorm_save8";
  const size_t count = rows * hidden;
  rra_status_t st = norm_common(bufs, outs, nranks, rows, hidden, gamma, dtype);
  if (st == RRA_SUCCESS && ((rows && (!codes || !scales || !rstd)) || !aligned(rstd, 4) || !(eps >= 0.f))) st = RRA_ERR_INVALID_ARG;
  if (st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, st);
  const size_t e = dtype == RRA_BFLOAT16 ? 2 : 4, S = count * e, nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  Ranges in, out;
  for (int r = 0; r < nranks; ++r) {
    in.push_back({bufs[r], S});
    out.push_back({outs[r], S});
  }
  in.push_back({gamma, hidden * e});
  out.push_back({codes, count});
  out.push_back({scales, rows * nblk});
  out.push_back({rstd, rows * 4});
  if (clash(in, out, nranks)) return done(call, nranks, count, dtype, 0, RRA_ERR_ALIAS);
  if (rows == 0) return done(call, nranks, 0, dtype, 0, RRA_SUCCESS);
  const bool vec = norm_vec(bufs, (const void* const*)outs, nranks, gamma, codes, hidden, e);
  const cudaError_t err = launch_norm_save8(nranks, dtype, vec, bufs, outs, gamma, rows, hidden, eps, codes, scales,
                                            rstd, reinterpret_cast<cudaStream_t>(stream));
  return done(call, nranks, count, dtype, 0, cuda_st(err));
}

rra_status_t rra_rmsnorm_restore8(const void* codes, const void* scales, const float* rstd, const void* gamma,
                                  void* out, size_t rows, size_t hidden, rra_dtype_t dtype, rra_stream_t stream) {
  const char* call = "rmsnorm_restore8";
  const size_t count = rows * hidden;
  const size_t e = dtype == RRA_BFLOAT16 ? 2 : 4;
  rra_status_t st = RRA_SUCCESS;
  if ((rows && (!codes || !scales || !out)) || hidden == 0 || (dtype != RRA_FLOAT32 && dtype != RRA_BFLOAT16) ||
      !aligned(out, e) || (gamma && !aligned(gamma, e)) || (rstd && !aligned(rstd, 4)))
    st = RRA_ERR_INVALID_ARG;
  else if (hidden > kNormMaxHidden || rows > 0x7FFFFFFFull)
    st = RRA_ERR_UNSUPPORTED;
  if (st != RRA_SUCCESS) return done(call, 1, count, dtype, 0, st);
  const size_t nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  if (clash({{codes, count}, {scales, rows * nblk}, {rstd, rstd ? rows * 4 : 0}, {gamma, gamma ? hidden * e : 0}},
            {{out, count * e}}))
    return done(call, 1, count, dtype, 0, RRA_ERR_ALIAS);
  if (rows == 0) return done(call, 1, 0, dtype, 0, RRA_SUCCESS);
  const void* o[1] = {out};
  const bool vec = norm_vec(nullptr, o, 1, gamma, codes, hidden, e);
  const cudaError_t err = launch_norm_restore8(dtype, vec, codes, scales, rstd, gamma, out, rows, hidden,
                                               reinterpret_cast<cudaStream_t>(stream));
  return done(call, 1, count, dtype, 0, cuda_st(err));
}

size_t rra_allreduce_rmsnorm_backward8_workspace_bytes(size_t rows, size_t hidden) {
  return up((size_t)norm_back8_ctas(rows) * norm_back8_pitch(hidden) * 4, kAlign);
}

rra_status_t rra_allreduce_rmsnorm_backward8(const void* const* grads, void* const* dxs, int nranks, size_t rows,
                                             size_t hidden, const void* codes, const void* scales,
                                             const float* rstd, const void* gamma, float* dgamma, void* workspace,
                                             size_t workspace_bytes, rra_dtype_t dtype, rra_stream_t stream) {
  const char* call = "allreduce_rmsnorm_backward8";
  const size_t count = rows * hidden;
  rra_status_t st = norm_common(grads, dxs, nranks, rows, hidden, gamma, dtype);
  const size_t need = rra_allreduce_rmsnorm_backward8_workspace_bytes(rows, hidden);
  if (st == RRA_SUCCESS && ((rows && (!codes || !scales || !rstd)) || !dgamma || !aligned(rstd, 4) || !aligned(dgamma, 4) ||
                            (need && !workspace) || !aligned(workspace, kAlign)))
    st = RRA_ERR_INVALID_ARG;
  if (st == RRA_SUCCESS && workspace_bytes < need) st = RRA_ERR_WORKSPACE;
  if (st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, st);
  const size_t e = dtype == RRA_BFLOAT16 ? 2 : 4, S = count * e, nblk = (hidden + kCkptBlock - 1) / kCkptBlock;
  Ranges in, out;
  for (int r = 0; r < nranks; ++r) {
    in.push_back({grads[r], S});
    out.push_back({dxs[r], S});
  }
  in.push_back({gamma, hidden * e});
  in.push_back({codes, count});
  in.push_back({scales, rows * nblk});
  in.push_back({rstd, rows * 4});
  out.push_back({dgamma, hidden * 4});
  out.push_back({workspace, need});
  if (clash(in, out, nranks)) return done(call, nranks, count, dtype, 0, RRA_ERR_ALIAS);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) return done(call, nranks, 0, dtype, 0, cuda_st(cudaMemsetAsync(dgamma, 0, hidden * 4, s)));
  const bool vec = norm_vec(grads, (const void* const*)dxs, nranks, gamma, codes, hidden, e);
  const cudaError_t err = launch_norm_back8(nranks, dtype, vec, grads, dxs, codes, scales, rstd, gamma, dgamma,
                                            static_cast<float*>(workspace), rows, hidden, s);
  return done(call, nranks, count, dtype, 0, cuda_st(err));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// gated feed-forward
// ---------------------------------------------------------------------------

namespace {

// Workspace of a call, in the order the call takes it.
// Few tokens go through the register-streamed product (kernels_skinny.cu): up
// to 8 always; 9 to 16, which it takes as two products per weight, where rows
// are whole 16-byte units and, for the loss (`logits`: elements of its
// weights), up to 2^27 weights (16 tokens, us, streamed against tiles: 8 x
// 1728 gated columns of hidden 5120 53 and 56, of 1024 11 and 14; 131072
// columns of hidden 1024 52 and 54, of 5120 228 and 208, of 1027 204 and 174).
bool skinny(size_t T, size_t D, size_t logits) {
  return T <= 8 || (T <= 16 && (D % 8 != 0 || logits <= (size_t)1 << 27));
}

// Whether the gated backward keeps what bfloat16 leaves of dg and du, as rows
// of their own behind the tokens': few entries' roundings do not average out
// (kernels_gated_ffn.cu), and both halves fit the 256 rows of dx's tile.
bool gate_rests(size_t T) { return T <= 128; }

size_t ffn_bytes(int n, size_t T, size_t D, size_t F, bool back) {
  Bump b{nullptr};
  if (padded(D) && (back || !skinny(T, D, 0))) {
    b.take(T * pad_ld(D) * 2);
    for (int i = 0; i < 2 * n; ++i) b.take(F * pad_ld(D) * 2);
  }
  if (back) {
    const bool two = gate_rests(T);
    const size_t rows = two ? 2 * T : T;
    for (int i = 0; i < 2 * n; ++i) b.take(rows * up(F, 64) * 2);
    const size_t kb = 2 * (size_t)n * ((F + 63) / 64);
    b.take(pick_split(rows, D, kb).slot_bytes);
    if (two) b.take(rows * slot_ld(D) * 4);
  }
  return b.at;
}

rra_status_t ffn_check(const void* x, const void* const* gates, const void* const* ups, const void* const* acts,
                       int n, size_t T, size_t D, size_t F, int act, int dt, const void* ws, size_t ws_bytes,
                       bool back) {
  if (n > kMaxRanks) return RRA_ERR_UNSUPPORTED;
  if (n < 1 || (T && !x) || !gates || !ups || !acts || D == 0 || (act != RRA_ACT_SILU && act != RRA_ACT_GELU_TANH))
    return RRA_ERR_INVALID_ARG;
  if (dt != RRA_BFLOAT16)
    return dt == RRA_FLOAT32 || dt == RRA_INT32 ? RRA_ERR_UNSUPPORTED : RRA_ERR_INVALID_ARG;
  if (bad_extent(T) || bad_extent(D) || bad_extent(F)) return RRA_ERR_UNSUPPORTED;
  if (T * D > SIZE_MAX / 1024 || T * F > SIZE_MAX / 1024 || F * D > SIZE_MAX / 1024) return RRA_ERR_UNSUPPORTED;
  if (too_many_tiles(T, 2 * F * n, 2 * n) || too_many_tiles(2 * F * n, D, 2 * n) || too_many_tiles(T, D, 0))
    return RRA_ERR_UNSUPPORTED;
  for (int r = 0; r < n; ++r) {
    if ((F && (!gates[r] || !ups[r])) || (T && F && !acts[r]) || !aligned(acts[r], 2) || !aligned(gates[r], 2) || !aligned(ups[r], 2))
      return RRA_ERR_INVALID_ARG;
    if (!aligned(gates[r], 16) || !aligned(ups[r], 16)) return RRA_ERR_UNSUPPORTED;
  }
  if (!aligned(x, 2)) return RRA_ERR_INVALID_ARG;
  if (!aligned(x, 16)) return RRA_ERR_UNSUPPORTED;
  const size_t need = ffn_bytes(n, T, D, F, back);
  if ((need && !ws) || !aligned(ws, kAlign)) return RRA_ERR_INVALID_ARG;
  if (ws_bytes < need) return RRA_ERR_WORKSPACE;
  return RRA_SUCCESS;
}

}  // namespace

extern "C" {

size_t rra_gated_ffn_workspace_bytes(int nranks, size_t tokens, size_t hidden, size_t width, int backward) {
  if (nranks < 1 || nranks > kMaxRanks) return 0;
  return ffn_bytes(nranks, tokens, hidden, width, backward != 0);
}

rra_status_t rra_gated_ffn(const void* x, const void* const* gates, const void* const* ups, void* const* acts,
                           int nranks, size_t tokens, size_t hidden, size_t width, rra_act_t act,
                           rra_dtype_t dtype, void* workspace, size_t workspace_bytes, rra_stream_t stream) {
  const char* call = "gated_ffn";
  const size_t T = tokens, D = hidden, F = width, count = T * F;
  rra_status_t st = ffn_check(x, gates, ups, (const void* const*)acts, nranks, T, D, F, act, dtype, workspace,
                              workspace_bytes, false);
  if (st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, st);
  Ranges in{{x, T * D * 2}}, out{{workspace, ffn_bytes(nranks, T, D, F, false)}};
  for (int r = 0; r < nranks; ++r) {
    in.push_back({gates[r], F * D * 2});
    in.push_back({ups[r], F * D * 2});
    out.push_back({acts[r], T * F * 2});
  }
  if (clash(in, out)) return done(call, nranks, count, dtype, 0, RRA_ERR_ALIAS);
  if (T == 0 || F == 0) return done(call, nranks, 0, dtype, 0, RRA_SUCCESS);
  if (!device_status()) return done(call, nranks, count, dtype, 0, RRA_ERR_NOT_INITIALIZED);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (skinny(T, D, 0)) {
    SkinnyArgs a{};
    a.x = x;
    a.tokens = (int)T;
    a.hidden = (int)D;
    a.width = (int)F;
    const size_t units = (size_t)nranks * (size_t)sk_gate_units((int)F, D % 8 == 0);
    if (units > INT_MAX / 2) return done(call, nranks, count, dtype, 0, RRA_ERR_UNSUPPORTED);
    a.units = (int)units;
    for (int r = 0; r < nranks; ++r) {
      a.w[2 * r] = gates[r];
      a.w[2 * r + 1] = ups[r];
      a.out[r] = acts[r];
    }
    int grid = 0;
    const cudaError_t e = launch_skinny_gate(a, act, s, &grid);
    return done(call, nranks, count, dtype, grid, cuda_st(e));
  }
  Bump ws{static_cast<char*>(workspace)};
  TcArgs args;
  TcArgs* const p = &args;
  clear(p);
  p->shape = pick_shape(T);
  Placer place(ws);
  const Mat X = place(x, T, D);
  bool ok = map_k(&p->a[0], X, p->shape.a_rows);
  for (int r = 0; r < nranks && ok; ++r) {
    const Mat G = place(gates[r], F, D), U = place(ups[r], F, D);
    ok = map_k(&p->b[2 * r], G) && map_k(&p->b[2 * r + 1], U);
    TcGroup g{};
    g.a = 0;
    g.b = 2 * r;
    g.M = (int)T;
    g.N = (int)F;
    g.out = acts[r];
    g.ld = (long long)F;
    g.vec = aligned(acts[r], 16) && F % 8 == 0;
    ok = ok && add_group(p, g, true);
  }
  if (!ok || !place.launch(s)) return done(call, nranks, count, dtype, 0, RRA_ERR_CUDA);
  one_k_axis(p, D);
  p->pair_b = 1;
  p->act = act;
  p->status = device_status();
  int grid = 0;
  const cudaError_t e = launch_tc_gate(*p, s, &grid);
  return done(call, nranks, count, dtype, grid, cuda_st(e));
}

rra_status_t rra_gated_ffn_backward(const void* x, const void* const* gates, const void* const* ups,
                                    const void* const* dacts, void* dx, void* const* dgates, void* const* dups,
                                    int nranks, size_t tokens, size_t hidden, size_t width, rra_act_t act,
                                    rra_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                    rra_stream_t stream) {
  const char* call = "gated_ffn_backward";
  const size_t T = tokens, D = hidden, F = width, count = T * F;
  rra_status_t st =
      ffn_check(x, gates, ups, dacts, nranks, T, D, F, act, dtype, workspace, workspace_bytes, true);
  if (st == RRA_SUCCESS && ((T && !dx) || !dgates || !dups || !aligned(dx, 2))) st = RRA_ERR_INVALID_ARG;
  for (int r = 0; r < nranks && st == RRA_SUCCESS; ++r)
    if ((F && (!dgates[r] || !dups[r])) || !aligned(dgates[r], 2) || !aligned(dups[r], 2)) st = RRA_ERR_INVALID_ARG;
  if (st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, st);
  Ranges in{{x, T * D * 2}}, out{{workspace, ffn_bytes(nranks, T, D, F, true)}, {dx, T * D * 2}};
  for (int r = 0; r < nranks; ++r) {
    in.push_back({gates[r], F * D * 2});
    in.push_back({ups[r], F * D * 2});
    in.push_back({dacts[r], T * F * 2});
    out.push_back({dgates[r], F * D * 2});
    out.push_back({dups[r], F * D * 2});
  }
  if (clash(in, out)) return done(call, nranks, count, dtype, 0, RRA_ERR_ALIAS);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0 || F == 0) {
    cudaError_t e = T ? cudaMemsetAsync(dx, 0, T * D * 2, s) : cudaSuccess;
    for (int r = 0; r < nranks && F && e == cudaSuccess; ++r) {
      e = cudaMemsetAsync(dgates[r], 0, F * D * 2, s);
      if (e == cudaSuccess) e = cudaMemsetAsync(dups[r], 0, F * D * 2, s);
    }
    return done(call, nranks, 0, dtype, 0, cuda_st(e));
  }
  if (!device_status()) return done(call, nranks, count, dtype, 0, RRA_ERR_NOT_INITIALIZED);
  Bump ws{static_cast<char*>(workspace)};
  Placer place(ws);
  const Mat X = place(x, T, D);
  Mat W[2 * kMaxRanks], dW[2 * kMaxRanks];
  for (int i = 0; i < 2 * nranks; ++i) W[i] = place(i % 2 ? ups[i / 2] : gates[i / 2], F, D);
  const bool two = gate_rests(T);
  const size_t ldf = up(F, 64), rows = two ? 2 * T : T;
  for (int i = 0; i < 2 * nranks; ++i) dW[i] = Mat{ws.take(rows * ldf * 2), rows, F, ldf};
  const size_t kb_seg = (F + 63) / 64, kb = 2 * (size_t)nranks * kb_seg;
  const Split sp = pick_split(rows, D, kb);
  float* slots = static_cast<float*>(ws.take(sp.slot_bytes));
  float* acc = two ? static_cast<float*>(ws.take(rows * slot_ld(D) * 4)) : nullptr;
  if (!place.launch(s)) return done(call, nranks, count, dtype, 0, RRA_ERR_CUDA);

  // dg, du
  TcArgs args;
  TcArgs* const p = &args;
  clear(p);
  p->shape = pick_shape(T);
  bool ok = map_k(&p->a[0], X, p->shape.a_rows);
  for (int r = 0; r < nranks && ok; ++r) {
    ok = map_k(&p->b[2 * r], W[2 * r]) && map_k(&p->b[2 * r + 1], W[2 * r + 1]);
    TcGroup g{};
    g.b = 2 * r;
    g.M = (int)T;
    g.N = (int)F;
    g.out = const_cast<void*>(dW[2 * r].p);
    g.out2 = const_cast<void*>(dW[2 * r + 1].p);
    g.ld = (long long)ldf;
    g.in = dacts[r];
    g.ld_in = (long long)F;
    g.vec = aligned(dacts[r], 16) && F % 8 == 0;
    ok = ok && add_group(p, g, true);
  }
  if (!ok) return done(call, nranks, count, dtype, 0, RRA_ERR_CUDA);
  one_k_axis(p, D);
  p->pair_b = 1;
  p->act = act;
  p->rest_row = two ? (int)T : 0;
  p->status = device_status();
  int grid = 0;
  cudaError_t e = launch_tc_gate_back(*p, s, &grid);
  if (e != cudaSuccess) return done(call, nranks, count, dtype, grid, RRA_ERR_CUDA);

  // dx: the shards' products as segments of one K axis; second halves are
  // rows of the same tile, added by the join
  clear(p);
  p->nsegs = 2 * nranks;
  for (int i = 0; i < 2 * nranks && ok; ++i) {
    ok = map_k(&p->a[i], dW[i]) && map_mn(&p->b[i], W[i]);
    p->seg_k0[i] = (int)(i * kb_seg);
  }
  p->kblocks = (int)kb;
  p->full = sp.full;
  p->splits = sp.splits;
  p->slots = slots;
  TcGroup g{};
  g.M = (int)rows;
  g.N = (int)D;
  g.ld = (long long)(two ? slot_ld(D) : D);
  g.out = two ? (void*)acc : dx;
  g.vec = two || (aligned(dx, 16) && D % 8 == 0);
  ok = ok && add_group(p, g, false);
  p->status = device_status();
  if (!ok) return done(call, nranks, count, dtype, 0, RRA_ERR_CUDA);
  e = launch_tc_input_grad(*p, two, s, &grid);
  if (e == cudaSuccess)
    e = launch_join_tiles({acc, slots, dx, (int)slot_ld(D), (int)T, (int)D, p->group[0].mt, p->group[0].nt, sp.full,
                           sp.splits, TcFix{}, two ? (int)T : 0}, s);
  if (e != cudaSuccess) return done(call, nranks, count, dtype, grid, RRA_ERR_CUDA);

  // dG, dU
  clear(p);
  ok = map_mn(&p->b[0], X);
  for (int i = 0; i < 2 * nranks && ok; ++i) {
    ok = map_mn(&p->a[i], dW[i]);
    void* o = i % 2 ? dups[i / 2] : dgates[i / 2];
    TcGroup h{};
    h.a = i;
    h.M = (int)F;
    h.N = (int)D;
    h.out = o;
    h.ld = (long long)D;
    h.vec = aligned(o, 16) && D % 8 == 0;
    ok = ok && add_group(p, h, false);
  }
  if (!ok) return done(call, nranks, count, dtype, 0, RRA_ERR_CUDA);
  token_axis(p, T, two);
  p->status = device_status();
  e = launch_tc_weight_grad(*p, s, &grid);
  return done(call, nranks, count, dtype, grid, cuda_st(e));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// vocabulary loss
// ---------------------------------------------------------------------------

namespace {

size_t vocab_tiles(int n, const size_t* vocab) {
  size_t t = 0;
  for (int r = 0; r < n; ++r) t += tiles256(vocab[r]);
  return t;
}

// Fixed part of a call's workspace: padded operands, and what forward or
// backward needs beside a piece.
struct LossPlan {
  size_t fixed = 0;        // bytes before the piece
  size_t rows = 0;         // rows of dl
  size_t piece_tiles = 0;  // 256-column tiles per piece
  Split split;             // of dx's tiles
  bool acc = false;        // dx is summed over pieces in float32
};

// Whether dl keeps what bfloat16 leaves of its entries, as rows of their own
// behind the tokens': a second block of 64 rows for the product of the
// weights' gradient, which takes one at the least.
bool rests(size_t T) { return T <= 32; }

// Blocks of 32 rows of the first n shards.
size_t blocks32(int n, const size_t* vocab) {
  size_t b = 0;
  for (int r = 0; r < n; ++r) b += (vocab[r] + 31) / 32;
  return b;
}

size_t vocab_rows(int n, const size_t* vocab) {
  size_t v = 0;
  for (int r = 0; r < n; ++r) v += vocab[r];
  return v;
}

long long skinny_units(int n, const size_t* vocab, size_t D) {
  long long u = 0;
  for (int r = 0; r < n; ++r) u += sk_loss_units((long long)vocab[r], D % 8 == 0);
  return u;
}

LossPlan loss_plan(int n, size_t T, size_t D, const size_t* vocab, bool back, size_t room) {
  LossPlan q;
  if (T == 0) return q;
  Bump b{nullptr};
  if (!back && skinny(T, D, vocab_rows(n, vocab) * D)) {
    b.take((size_t)skinny_most(skinny_units(n, vocab, D)) * T * sizeof(float2));
    b.take(T * 4);
    q.fixed = b.at;
    return q;
  }
  if (padded(D)) {
    b.take(T * pad_ld(D) * 2);
    for (int r = 0; r < n; ++r) b.take(vocab[r] * pad_ld(D) * 2);
  }
  if (back) {
    b.take(T * sizeof(float4));
    for (int i = 0; i < 4; ++i) b.take(T * 4);
    b.take((blocks32(n, vocab) + 1) * 4);
  }
  const size_t tiles = vocab_tiles(n, vocab);
  if (!back) {
    b.take(2 * tiles * T * sizeof(float2));
    b.take(T * 4);
    q.fixed = b.at;
    return q;
  }
  q.rows = rests(T) ? 2 * T : T;
  const size_t col = q.rows * 512;  // bytes of a tile column of dl
  const size_t base = b.at;
  // the parts of dx's K axis depend on the piece, which depends on the room
  // their slots leave: take the largest piece that fits with its own slots
  size_t piece = std::max<size_t>(1, std::min(tiles, kPieceBytes / std::max<size_t>(col, 1)));
  for (;; --piece) {
    q.split = pick_split(T, D, piece * 4);
    q.acc = piece < tiles;
    q.fixed = base + up(q.split.slot_bytes, kAlign) + (q.acc ? up(T * slot_ld(D) * 4, kAlign) : 0);
    q.piece_tiles = piece;
    if (piece == 1 || room == SIZE_MAX || q.fixed + piece * col <= room) break;
    // jump to what the room allows at most
    const size_t most = room > q.fixed ? (room - q.fixed) / col : 0;
    if (most < piece - 1) piece = std::max<size_t>(most, 1) + 1;
  }
  return q;
}

rra_status_t loss_check(const void* x, const void* const* weights, const size_t* vocab, const void* targets, int n,
                        size_t T, size_t D, int dt, const void* ws, size_t* total) {
  if (n > kMaxRanks) return RRA_ERR_UNSUPPORTED;
  if (n < 1 || !weights || !vocab || (T && (!x || !targets)) || D == 0) return RRA_ERR_INVALID_ARG;
  if (dt != RRA_BFLOAT16)
    return dt == RRA_FLOAT32 || dt == RRA_INT32 ? RRA_ERR_UNSUPPORTED : RRA_ERR_INVALID_ARG;
  if (bad_extent(T) || bad_extent(D)) return RRA_ERR_UNSUPPORTED;
  size_t V = 0;
  for (int r = 0; r < n; ++r) {
    if (bad_extent(vocab[r])) return RRA_ERR_UNSUPPORTED;
    V += vocab[r];
    if (vocab[r] && (!weights[r] || !aligned(weights[r], 2))) return RRA_ERR_INVALID_ARG;
    if (vocab[r] && !aligned(weights[r], 16)) return RRA_ERR_UNSUPPORTED;
  }
  if (V == 0 || !aligned(x, 2) || !aligned(targets, 8) || !aligned(ws, kAlign)) return RRA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || bad_extent(V)) return RRA_ERR_UNSUPPORTED;
  if (T * D > SIZE_MAX / 1024 || V * D > SIZE_MAX / 1024 || too_many_tiles(T, V, n) || too_many_tiles(V, D, n) ||
      too_many_tiles(T, D, 0))
    return RRA_ERR_UNSUPPORTED;
  *total = V;
  return RRA_SUCCESS;
}

}  // namespace

extern "C" {

size_t rra_vocab_loss_workspace_bytes(int nranks, size_t tokens, size_t hidden, const size_t* vocab, int backward) {
  if (nranks < 1 || nranks > kMaxRanks || !vocab) return 0;
  const LossPlan q = loss_plan(nranks, tokens, hidden, vocab, backward != 0, backward == 2 ? 0 : SIZE_MAX);
  return q.fixed + up(q.piece_tiles * q.rows * 512, kAlign);
}

rra_status_t rra_vocab_loss(const void* x, const void* const* weights, const size_t* vocab, const int64_t* targets,
                            int nranks, size_t tokens, size_t hidden, int64_t ignore_index, float* loss,
                            float* lse, rra_dtype_t dtype, void* workspace, size_t workspace_bytes,
                            rra_stream_t stream) {
  const char* call = "vocab_loss";
  const size_t T = tokens, D = hidden;
  size_t V = 0;
  rra_status_t st = loss_check(x, weights, vocab, targets, nranks, T, D, dtype, workspace, &V);
  if (st == RRA_SUCCESS && ((T && (!loss || !lse)) || !aligned(loss, 4) || !aligned(lse, 4))) st = RRA_ERR_INVALID_ARG;
  if (st != RRA_SUCCESS) return done(call, nranks, T * V, dtype, 0, st);
  const size_t need = loss_plan(nranks, T, D, vocab, false, SIZE_MAX).fixed;
  if (need && !workspace) return done(call, nranks, T * V, dtype, 0, RRA_ERR_INVALID_ARG);
  if (workspace_bytes < need) return done(call, nranks, T * V, dtype, 0, RRA_ERR_WORKSPACE);
  Ranges in{{x, T * D * 2}, {targets, T * 8}}, out{{workspace, need}, {loss, T * 4}, {lse, T * 4}};
  for (int r = 0; r < nranks; ++r) in.push_back({weights[r], vocab[r] * D * 2});
  if (clash(in, out)) return done(call, nranks, T * V, dtype, 0, RRA_ERR_ALIAS);
  if (T == 0) return done(call, nranks, 0, dtype, 0, RRA_SUCCESS);
  if (!device_status()) return done(call, nranks, T * V, dtype, 0, RRA_ERR_NOT_INITIALIZED);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Bump ws{static_cast<char*>(workspace)};
  if (skinny(T, D, V * D)) {
    SkinnyArgs a{};
    a.x = x;
    a.tokens = (int)T;
    a.hidden = (int)D;
    long long col = 0;
    for (int r = 0; r < nranks; ++r) {
      a.w[r] = weights[r];
      a.rows[r] = (long long)vocab[r];
      a.col0[r] = col;
      a.unit0[r + 1] = a.unit0[r] + (int)sk_loss_units((long long)vocab[r], D % 8 == 0);
      col += (long long)vocab[r];
    }
    a.units = a.unit0[nranks];
    for (int r = nranks; r < kMaxRanks; ++r) a.unit0[r + 1] = a.units;
    a.targets = reinterpret_cast<const long long*>(targets);
    a.ignore_index = ignore_index;
    a.part = static_cast<float2*>(ws.take((size_t)skinny_most(a.units) * T * sizeof(float2)));
    a.hit = static_cast<float*>(ws.take(T * 4));
    int grid = 0;
    cudaError_t e = launch_skinny_lse(a, s, &grid);
    if (e == cudaSuccess)
      e = launch_loss_join(a.part, grid, a.hit, a.targets, ignore_index, x, weights, vocab, nranks, D, (int)T, loss,
                           lse, s);
    return done(call, nranks, T * V, dtype, grid, cuda_st(e));
  }
  TcArgs args;
  TcArgs* const p = &args;
  clear(p);
  p->shape = pick_shape(T);
  Placer place(ws);
  const Mat X = place(x, T, D);
  bool ok = map_k(&p->a[0], X, p->shape.a_rows);
  long long col0 = 0;
  int parts = 0;
  for (int r = 0; r < nranks && ok; ++r) {
    if (vocab[r]) {
      const Mat W = place(weights[r], vocab[r], D);
      ok = map_k(&p->b[r], W);
      TcGroup g{};
      g.b = r;
      g.M = (int)T;
      g.N = (int)vocab[r];
      g.col0 = col0;
      g.part0 = parts;
      ok = ok && add_group(p, g, false);
    }
    col0 += (long long)vocab[r];
    parts += (int)tiles256(vocab[r]);
  }
  if (!ok || !place.launch(s)) return done(call, nranks, T * V, dtype, 0, RRA_ERR_CUDA);
  one_k_axis(p, D);
  p->part = static_cast<float2*>(ws.take(2 * (size_t)parts * T * sizeof(float2)));
  p->part_ld = (long long)T;
  p->hit = static_cast<float*>(ws.take(T * 4));
  p->targets = reinterpret_cast<const long long*>(targets);
  p->ignore_index = ignore_index;
  p->status = device_status();
  int grid = 0;
  cudaError_t e = launch_tc_lse(*p, s, &grid);
  if (e == cudaSuccess)
    e = launch_loss_join(p->part, 2 * parts, p->hit, p->targets, ignore_index, x, weights, vocab, nranks, D, (int)T,
                         loss, lse, s);
  return done(call, nranks, T * V, dtype, grid, cuda_st(e));
}

rra_status_t rra_vocab_loss_backward(const void* x, const void* const* weights, const size_t* vocab,
                                     const int64_t* targets, const float* lse, const float* grad_loss, void* dx,
                                     void* const* dweights, int nranks, size_t tokens, size_t hidden,
                                     int64_t ignore_index, rra_dtype_t dtype, void* workspace,
                                     size_t workspace_bytes, rra_stream_t stream) {
  const char* call = "vocab_loss_backward";
  const size_t T = tokens, D = hidden;
  size_t V = 0;
  rra_status_t st = loss_check(x, weights, vocab, targets, nranks, T, D, dtype, workspace, &V);
  if (st == RRA_SUCCESS && ((T && (!lse || !grad_loss || !dx)) || !dweights || !aligned(lse, 4) || !aligned(grad_loss, 4) ||
                            !aligned(dx, 2)))
    st = RRA_ERR_INVALID_ARG;
  for (int r = 0; r < nranks && st == RRA_SUCCESS; ++r)
    if (vocab[r] && (!dweights[r] || !aligned(dweights[r], 2))) st = RRA_ERR_INVALID_ARG;
  if (st != RRA_SUCCESS) return done(call, nranks, T * V, dtype, 0, st);
  if (T && !workspace) return done(call, nranks, T * V, dtype, 0, RRA_ERR_INVALID_ARG);
  const LossPlan q = loss_plan(nranks, T, D, vocab, true, workspace_bytes);
  const size_t need = q.fixed + q.piece_tiles * q.rows * 512;
  if (workspace_bytes < need) return done(call, nranks, T * V, dtype, 0, RRA_ERR_WORKSPACE);
  Ranges in{{x, T * D * 2}, {targets, T * 8}, {lse, T * 4}, {grad_loss, T * 4}},
      out{{workspace, need}, {dx, T * D * 2}};
  for (int r = 0; r < nranks; ++r) {
    in.push_back({weights[r], vocab[r] * D * 2});
    out.push_back({vocab[r] ? dweights[r] : nullptr, vocab[r] * D * 2});
  }
  if (clash(in, out)) return done(call, nranks, T * V, dtype, 0, RRA_ERR_ALIAS);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    cudaError_t e = cudaSuccess;
    for (int r = 0; r < nranks && e == cudaSuccess; ++r)
      if (vocab[r]) e = cudaMemsetAsync(dweights[r], 0, vocab[r] * D * 2, s);
    return done(call, nranks, 0, dtype, 0, cuda_st(e));
  }
  if (!device_status()) return done(call, nranks, T * V, dtype, 0, RRA_ERR_NOT_INITIALIZED);

  Bump ws{static_cast<char*>(workspace)};
  Placer place(ws);
  const Mat X = place(x, T, D);
  Mat W[kMaxRanks];
  for (int r = 0; r < nranks; ++r) W[r] = place(weights[r], vocab[r], D);
  float4* rows = static_cast<float4*>(ws.take(T * sizeof(float4)));
  TcFix fix{};
  int* column = static_cast<int*>(ws.take(T * 4));
  float* rest = static_cast<float*>(ws.take(T * 4));
  int* token = static_cast<int*>(ws.take(T * 4));
  int* sorted = static_cast<int*>(ws.take(T * 4));
  int* start = static_cast<int*>(ws.take((blocks32(nranks, vocab) + 1) * 4));
  fix.column = column;
  fix.lo = rest;
  fix.start = start;
  fix.token = token;
  fix.sorted = sorted;
  bool ok = place.launch(s) &&
            launch_loss_rows(x, weights, vocab, nranks, D, (int)T, reinterpret_cast<const long long*>(targets),
                             ignore_index, lse, grad_loss, rows, column, rest, start, token, sorted,
                             s) == cudaSuccess;
  if (!ok) return done(call, nranks, T * V, dtype, 0, RRA_ERR_CUDA);
  float* slots = static_cast<float*>(ws.take(q.split.slot_bytes));
  float* acc = q.acc ? static_cast<float*>(ws.take(T * slot_ld(D) * 4)) : nullptr;
  char* dl = ws.base + ws.at;
  const size_t ld = q.piece_tiles * 256;

  // dx's additions are made where a tile is rounded: in the join, or in the
  // product's own epilogue for tiles of a single piece that take the whole K
  // axis
  TcFix dx_fix = fix;
  dx_fix.kind = 1;
  dx_fix.ld = (long long)X.ld;
  for (int r = 0; r < nranks; ++r) {
    dx_fix.w[r] = W[r].p;
    dx_fix.first[r + 1] = dx_fix.first[r] + (long long)vocab[r];
  }

  TcArgs args;
  TcArgs* const p = &args;
  const size_t tiles = vocab_tiles(nranks, vocab);
  int grid = 0;
  cudaError_t e = cudaSuccess;
  for (size_t t0 = 0; t0 < tiles && e == cudaSuccess; t0 += q.piece_tiles) {
    const size_t t1 = std::min(tiles, t0 + q.piece_tiles);
    // the shards' rows [lo, hi) inside this piece, and their columns of dl
    size_t lo[kMaxRanks], hi[kMaxRanks], at[kMaxRanks], tile = 0, col = 0;
    long long first[kMaxRanks];
    for (int r = 0; r < nranks; ++r) {
      const size_t nt = tiles256(vocab[r]);
      const size_t a = std::min(std::max(t0, tile), tile + nt) - tile, b = std::min(std::max(t1, tile), tile + nt) - tile;
      lo[r] = std::min(vocab[r], a * 256);
      hi[r] = std::min(vocab[r], b * 256);
      at[r] = (tile + a >= t0 ? tile + a - t0 : 0) * 256;
      first[r] = (long long)(col + lo[r]);
      tile += nt;
      col += vocab[r];
    }
    // dl of the piece
    clear(p);
    p->shape = pick_shape(T);
    ok = map_k(&p->a[0], X, p->shape.a_rows);
    for (int r = 0; r < nranks && ok; ++r) {
      if (hi[r] <= lo[r]) continue;
      ok = map_k(&p->b[r], W[r]);
      TcGroup g{};
      g.b = r;
      g.M = (int)T;
      g.N = (int)(hi[r] - lo[r]);
      g.n0 = (int)lo[r];
      g.col0 = first[r];
      g.out = dl + at[r] * 2;
      g.ld = (long long)ld;
      ok = ok && add_group(p, g, false);
    }
    if (!ok) return done(call, nranks, T * V, dtype, 0, RRA_ERR_CUDA);
    one_k_axis(p, D);
    p->targets = reinterpret_cast<const long long*>(targets);
    p->rows = rows;
    p->rest_row = rests(T) ? (int)T : 0;
    p->status = device_status();
    e = launch_tc_dlogits(*p, s, &grid);
    if (e != cudaSuccess) break;

    // dx (+)= dl W over the piece
    clear(p);
    size_t kb = 0;
    for (int r = 0; r < nranks && ok; ++r) {
      if (hi[r] <= lo[r]) continue;
      const Mat A{dl + at[r] * 2, T, hi[r] - lo[r], ld};
      const Mat B{static_cast<const char*>(W[r].p) + lo[r] * W[r].ld * 2, hi[r] - lo[r], D, W[r].ld};
      ok = map_k(&p->a[p->nsegs], A) && map_mn(&p->b[p->nsegs], B);
      p->seg_k0[p->nsegs++] = (int)kb;
      kb += (hi[r] - lo[r] + 63) / 64;
    }
    if (p->nsegs == 1) {  // one segment is walked as a plain K axis of group 0
      p->seg_k0[0] = 0;
    }
    p->kblocks = (int)kb;
    p->full = q.split.full;
    p->splits = q.split.splits;
    p->slots = slots;
    p->accumulate = t0 > 0;
    p->fix = dx_fix;
    TcGroup g{};
    g.M = (int)T;
    g.N = (int)D;
    g.ld = (long long)(acc ? slot_ld(D) : D);
    g.out = acc ? (void*)acc : dx;
    g.vec = acc || (aligned(dx, 16) && D % 8 == 0);
    ok = ok && add_group(p, g, false);
    p->status = device_status();
    if (!ok) return done(call, nranks, T * V, dtype, 0, RRA_ERR_CUDA);
    e = launch_tc_input_grad(*p, q.acc, s, &grid);
    if (e != cudaSuccess) break;

    // dW of the piece's rows
    clear(p);
    p->fix = fix;
    p->fix.kind = 2;
    p->fix.w[0] = X.p;
    p->fix.ld = (long long)X.ld;
    ok = map_mn(&p->b[0], X);
    for (int r = 0; r < nranks && ok; ++r) {
      if (hi[r] <= lo[r]) continue;
      const Mat A{dl + at[r] * 2, q.rows, hi[r] - lo[r], ld};
      ok = map_mn(&p->a[r], A);
      TcGroup h{};
      h.a = r;
      h.col0 = first[r];
      h.part0 = (int)(blocks32(r, vocab) + lo[r] / 32);
      h.M = (int)(hi[r] - lo[r]);
      h.N = (int)D;
      h.ld = (long long)D;
      h.out = static_cast<char*>(dweights[r]) + lo[r] * D * 2;
      h.vec = aligned(h.out, 16) && D % 8 == 0;
      ok = ok && add_group(p, h, false);
    }
    if (!ok) return done(call, nranks, T * V, dtype, 0, RRA_ERR_CUDA);
    token_axis(p, T, rests(T));
    p->status = device_status();
    e = launch_tc_weight_grad(*p, s, &grid);
  }
  if (e == cudaSuccess)
    e = launch_join_tiles({acc, slots, dx, (int)slot_ld(D), (int)T, (int)D, (int)tiles256(T), (int)tiles256(D),
                           q.split.full, q.split.splits, dx_fix}, s);
  return done(call, nranks, T * V, dtype, grid, cuda_st(e));
}

}  // extern "C"
