// rra_serve.cpp -- the C ABI of the serving-step operators: argument checks,
// tensor maps and launches.  All computation runs in kernels_mx4.cu,
// kernels_mx4_product.cu, kernels_mx4_few.cu and kernels_vocab_sample.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>

#include "abi_util.h"
#include "rra.h"
#include "rra_internal.h"
#include "serve_host.h"

using namespace rra;

namespace {

size_t mx_blocks(size_t cols) { return (cols + 31) / 32; }
size_t mx_across(size_t cols) { return (cols + 127) / 128; }
size_t mx_bands(size_t rows) { return (rows + 127) / 128; }
size_t mx_row_bytes(size_t cols) { return 16 * mx_blocks(cols); }
size_t mx_scale_bytes(size_t rows, size_t cols) { return mx_bands(rows) * mx_across(cols) * 512; }

bool bad_extent(size_t a) { return a > (size_t)INT_MAX - 1024; }
bool bad_matrix(size_t rows, size_t cols) {
  return bad_extent(rows) || bad_extent(cols) || (cols && rows > SIZE_MAX / 1024 / cols);
}
bool float_type(int dt) { return dt == RRA_FLOAT32 || dt == RRA_BFLOAT16; }
size_t size_of(int dt) { return dt == RRA_BFLOAT16 ? 2 : 4; }

// An MX4 matrix of a call: both parts there, on 16 bytes.
rra_status_t mx_check(const rra_mx4_t& m, size_t rows, size_t cols) {
  if (rows && cols && (!m.codes || !m.scales)) return RRA_ERR_INVALID_ARG;
  return aligned(m.codes, 16) && aligned(m.scales, 16) ? RRA_SUCCESS : RRA_ERR_UNSUPPORTED;
}

void mx_ranges(Ranges& r, const rra_mx4_t& m, size_t rows, size_t cols) {
  r.push_back({m.codes, rows * mx_row_bytes(cols)});
  r.push_back({m.scales, mx_scale_bytes(rows, cols)});
}

// The first failure of several checks.
struct First {
  rra_status_t st = RRA_SUCCESS;
  void operator()(rra_status_t s) {
    if (st == RRA_SUCCESS) st = s;
  }
  void operator()(bool bad, rra_status_t s) {
    if (bad) (*this)(s);
  }
};

bool map_mx(CUtensorMap* codes, CUtensorMap* scales, const rra_mx4_t& m, size_t rows, size_t cols, int box_rows,
            int box_bands) {
  return mx4_map_codes(codes, m.codes, mx_row_bytes(cols), rows, box_rows) &&
         mx4_map_scales(scales, m.scales, mx_across(cols), mx_bands(rows), box_bands);
}

// How a call of these tokens is tiled: the few-token kernel takes weights as
// 128-row tiles, the other 256 (gated: 128 of each projection), tokens by 128 a
// CTA.
struct Plan {
  bool few, gated;
  int x_box, w_bands;
  size_t tile;  // weight rows (gated: of each projection)
  Plan(size_t tokens, size_t rows, bool g) : few(tokens <= mx4_few_most(rows, g)), gated(g) {
    x_box = few ? mx4_few_tile(tokens) : 128;
    tile = few || gated ? 128 : 256;
    w_bands = few || gated ? 1 : 2;
  }
  size_t tiles(size_t rows) const { return (rows + tile - 1) / tile; }
};

int k_tiles(size_t cols) { return (int)((cols + kMxKTile - 1) / kMxKTile); }

void start(Mx4Args* p, size_t tokens) {
  *p = Mx4Args{};
  p->tokens = (int)tokens;
  p->mt = (int)((tokens + 255) / 256);
  p->status = device_status();
}

void one_segment(Mx4Args* p, size_t cols) {
  p->nsegs = 1;
  p->seg_k0[0] = 0;
  p->kblocks = k_tiles(cols);
}

cudaError_t launch(Mx4Args* p, const Plan& plan, cudaStream_t s, int* grid) {
  return plan.few ? launch_mx4_few(*p, plan.gated, s, grid) : launch_mx4_product(*p, plan.gated, s, grid);
}

bool too_many(size_t tokens, size_t tiles) { return ((tokens + 255) / 256) * tiles > (size_t)INT_MAX / 4; }

}  // namespace

extern "C" {

size_t rra_mx4_scale_bytes(size_t rows, size_t cols) { return mx_scale_bytes(rows, cols); }

rra_status_t rra_mx4_quantize(const void* x, const rra_mx4_t* out, size_t rows, size_t cols, rra_dtype_t dtype,
                              rra_stream_t stream) {
  const char* call = "mx4_quantize";
  const size_t count = rows * cols;
  First f;
  f(!out || !float_type(dtype) || (rows && cols && !x) || (float_type(dtype) && !aligned(x, size_of(dtype))),
    RRA_ERR_INVALID_ARG);
  f(bad_matrix(rows, cols), RRA_ERR_UNSUPPORTED);
  if (f.st == RRA_SUCCESS) f(mx_check(*out, rows, cols));
  if (f.st != RRA_SUCCESS) return done(call, 1, count, dtype, 0, f.st);
  const size_t e = size_of(dtype);
  Ranges o;
  mx_ranges(o, *out, rows, cols);
  if (clash({{x, count * e}}, o)) return done(call, 1, count, dtype, 0, RRA_ERR_ALIAS);
  if (count == 0) return done(call, 1, 0, dtype, 0, RRA_SUCCESS);
  const bool vec = aligned(x, 16) && (cols * e) % 16 == 0;
  const cudaError_t err = launch_mx4_quantize(dtype, vec, x, out->codes, out->scales, rows, cols,
                                              reinterpret_cast<cudaStream_t>(stream));
  return done(call, 1, count, dtype, 0, cuda_st(err));
}

rra_status_t rra_mx4_restore(const rra_mx4_t* in, void* out, size_t rows, size_t cols, rra_dtype_t dtype,
                             rra_stream_t stream) {
  const char* call = "mx4_restore";
  const size_t count = rows * cols;
  First f;
  f(!in || !float_type(dtype) || (rows && cols && !out) || (float_type(dtype) && !aligned(out, size_of(dtype))),
    RRA_ERR_INVALID_ARG);
  f(bad_matrix(rows, cols), RRA_ERR_UNSUPPORTED);
  if (f.st == RRA_SUCCESS) f(mx_check(*in, rows, cols));
  if (f.st != RRA_SUCCESS) return done(call, 1, count, dtype, 0, f.st);
  const size_t e = size_of(dtype);
  Ranges i;
  mx_ranges(i, *in, rows, cols);
  if (clash(i, {{out, count * e}})) return done(call, 1, count, dtype, 0, RRA_ERR_ALIAS);
  if (count == 0) return done(call, 1, 0, dtype, 0, RRA_SUCCESS);
  const bool vec = aligned(out, 16) && (cols * e) % 16 == 0;
  const cudaError_t err = launch_mx4_restore(dtype, vec, in->codes, in->scales, out, rows, cols,
                                             reinterpret_cast<cudaStream_t>(stream));
  return done(call, 1, count, dtype, 0, cuda_st(err));
}

rra_status_t rra_allreduce_rmsnorm_mx4(const void* const* bufs, int nranks, size_t rows, size_t hidden,
                                       const void* gamma, float eps, const void* residual, void* residual_out,
                                       const rra_mx4_t* out, rra_dtype_t dtype, rra_stream_t stream) {
  const char* call = "allreduce_rmsnorm_mx4";
  const size_t count = rows * hidden;
  First f;
  f(nranks > kMaxRanks, RRA_ERR_UNSUPPORTED);
  f(!bufs || nranks < 1 || !gamma || !out || !float_type(dtype) || hidden == 0 || !(eps >= 0.f), RRA_ERR_INVALID_ARG);
  f(hidden > kNormMaxHidden || rows > 0x7FFFFFFFull, RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, f.st);
  const size_t e = size_of(dtype), S = count * e;
  f(!aligned(gamma, e) || !aligned(residual, e) || !aligned(residual_out, e), RRA_ERR_INVALID_ARG);
  bool vec = aligned(gamma, 16) && aligned(residual, 16) && aligned(residual_out, 16) && (hidden * e) % 16 == 0;
  Ranges in, o;
  in.push_back({residual, residual ? S : 0});  // residual_out may be residual
  o.push_back({residual_out, residual_out ? S : 0});
  for (int r = 0; r < nranks; ++r) {
    f((rows && !bufs[r]) || !aligned(bufs[r], e), RRA_ERR_INVALID_ARG);
    vec = vec && aligned(bufs[r], 16);
    in.push_back({bufs[r], S});
  }
  in.push_back({gamma, hidden * e});
  f(mx_check(*out, rows, hidden));
  if (f.st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, f.st);
  mx_ranges(o, *out, rows, hidden);
  if (clash(in, o, 1)) return done(call, nranks, count, dtype, 0, RRA_ERR_ALIAS);
  if (rows == 0) return done(call, nranks, 0, dtype, 0, RRA_SUCCESS);
  const cudaError_t err = launch_norm_mx4(nranks, dtype, vec, bufs, residual, residual_out, gamma, rows, hidden, eps,
                                          out->codes, out->scales, reinterpret_cast<cudaStream_t>(stream));
  return done(call, nranks, count, dtype, 0, cuda_st(err));
}

rra_status_t rra_mx4_product(const rra_mx4_t* x, const rra_mx4_t* weights, void* const* outs, int nranks,
                             size_t tokens, size_t hidden, const size_t* widths, rra_dtype_t dtype,
                             rra_stream_t stream) {
  const char* call = "mx4_product";
  const size_t T = tokens, D = hidden;
  First f;
  f(nranks > kMaxRanks, RRA_ERR_UNSUPPORTED);
  f(!x || !weights || !outs || !widths || nranks < 1 || D == 0 || !float_type(dtype), RRA_ERR_INVALID_ARG);
  f(bad_matrix(T, D), RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, 0, dtype, 0, f.st);
  const size_t e = size_of(dtype);
  for (int r = 0; r < nranks; ++r) f(bad_matrix(widths[r], D) || bad_matrix(T, widths[r]), RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, 0, dtype, 0, f.st);
  size_t rows = 0;
  for (int r = 0; r < nranks; ++r) rows += widths[r];
  const Plan plan(T, rows, false);
  f(mx_check(*x, T, D));
  Ranges in, o;
  mx_ranges(in, *x, T, D);
  size_t tiles = 0, count = 0;
  for (int r = 0; r < nranks; ++r) {
    f((T && widths[r] && !outs[r]) || !aligned(outs[r], e), RRA_ERR_INVALID_ARG);
    f(mx_check(weights[r], widths[r], D));
    mx_ranges(in, weights[r], widths[r], D);
    o.push_back({outs[r], T * widths[r] * e});
    tiles += plan.tiles(widths[r]);
    count += T * widths[r];
  }
  f(too_many(T, tiles), RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, f.st);
  if (clash(in, o)) return done(call, nranks, count, dtype, 0, RRA_ERR_ALIAS);
  if (count == 0) return done(call, nranks, 0, dtype, 0, RRA_SUCCESS);
  if (!device_status()) return done(call, nranks, count, dtype, 0, RRA_ERR_NOT_INITIALIZED);
  Mx4Args args;
  Mx4Args* const p = &args;
  start(p, T);
  one_segment(p, D);
  p->f32 = dtype == RRA_FLOAT32;
  bool ok = map_mx(&p->x[0], &p->xs[0], *x, T, D, plan.x_box, 1);
  for (int r = 0; r < nranks && ok; ++r) {
    if (widths[r] == 0) continue;
    ok = map_mx(&p->w[r], &p->ws[r], weights[r], widths[r], D, 128, plan.w_bands);
    Mx4Group& g = p->group[p->ngroups++];
    g.tile0 = p->tiles;
    g.tiles = (int)plan.tiles(widths[r]);
    g.rows = (int)widths[r];
    g.w = r;
    g.out = outs[r];
    g.ld = (long long)widths[r];
    g.vec = aligned(outs[r], 16) && (widths[r] * e) % 16 == 0;
    p->tiles += g.tiles;
  }
  if (!ok) return done(call, nranks, count, dtype, 0, RRA_ERR_CUDA);
  int grid = 0;
  const cudaError_t err = launch(p, plan, reinterpret_cast<cudaStream_t>(stream), &grid);
  return done(call, nranks, count, dtype, grid, cuda_st(err));
}

rra_status_t rra_mx4_product_sum(const rra_mx4_t* xs, const rra_mx4_t* weights, void* out, int nranks, size_t tokens,
                                 size_t width, size_t hidden, rra_dtype_t dtype, rra_stream_t stream) {
  const char* call = "mx4_product_sum";
  const size_t T = tokens, F = width, D = hidden, count = T * D;
  First f;
  f(nranks > kMaxRanks, RRA_ERR_UNSUPPORTED);
  f(!xs || !weights || nranks < 1 || !float_type(dtype) || (T && D && !out), RRA_ERR_INVALID_ARG);
  f(bad_matrix(T, F) || bad_matrix(D, F) || bad_matrix(T, D) || (F + kMxKTile) * (size_t)kMaxRanks > (size_t)INT_MAX,
    RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, f.st);
  const size_t e = size_of(dtype);
  const Plan plan(T, D, false);
  f(!aligned(out, e), RRA_ERR_INVALID_ARG);
  Ranges in;
  for (int r = 0; r < nranks; ++r) {
    f(mx_check(xs[r], T, F));
    f(mx_check(weights[r], D, F));
    mx_ranges(in, xs[r], T, F);
    mx_ranges(in, weights[r], D, F);
  }
  f(too_many(T, plan.tiles(D)), RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, count, dtype, 0, f.st);
  if (clash(in, {{out, count * e}})) return done(call, nranks, count, dtype, 0, RRA_ERR_ALIAS);
  if (count == 0) return done(call, nranks, 0, dtype, 0, RRA_SUCCESS);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (F == 0) return done(call, nranks, count, dtype, 0, cuda_st(cudaMemsetAsync(out, 0, count * e, s)));
  if (!device_status()) return done(call, nranks, count, dtype, 0, RRA_ERR_NOT_INITIALIZED);
  Mx4Args args;
  Mx4Args* const p = &args;
  start(p, T);
  p->f32 = dtype == RRA_FLOAT32;
  p->nsegs = nranks;
  bool ok = true;
  for (int r = 0; r < nranks && ok; ++r) {
    ok = map_mx(&p->x[r], &p->xs[r], xs[r], T, F, plan.x_box, 1) &&
         map_mx(&p->w[r], &p->ws[r], weights[r], D, F, 128, plan.w_bands);
    p->seg_k0[r] = p->kblocks;
    p->kblocks += k_tiles(F);
  }
  if (!ok) return done(call, nranks, count, dtype, 0, RRA_ERR_CUDA);
  Mx4Group& g = p->group[p->ngroups++];
  g.tiles = p->tiles = (int)plan.tiles(D);
  g.rows = (int)D;
  g.out = out;
  g.ld = (long long)D;
  g.vec = aligned(out, 16) && (D * e) % 16 == 0;
  int grid = 0;
  const cudaError_t err = launch(p, plan, s, &grid);
  return done(call, nranks, count, dtype, grid, cuda_st(err));
}

rra_status_t rra_mx4_gated_ffn(const rra_mx4_t* x, const rra_mx4_t* gates, const rra_mx4_t* ups,
                               const rra_mx4_t* acts, int nranks, size_t tokens, size_t hidden, size_t width,
                               rra_act_t act, rra_stream_t stream) {
  const char* call = "mx4_gated_ffn";
  const int dt = RRA_BFLOAT16;  // of the record only
  const size_t T = tokens, D = hidden, F = width, count = T * F;
  First f;
  f(nranks > kMaxRanks, RRA_ERR_UNSUPPORTED);
  f(!x || !gates || !ups || !acts || nranks < 1 || D == 0 || (act != RRA_ACT_SILU && act != RRA_ACT_GELU_TANH),
    RRA_ERR_INVALID_ARG);
  f(bad_matrix(T, D) || bad_matrix(F, D) || bad_matrix(T, F), RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, count, dt, 0, f.st);
  const Plan plan(T, F * nranks, true);
  f(mx_check(*x, T, D));
  Ranges in, o;
  mx_ranges(in, *x, T, D);
  for (int r = 0; r < nranks; ++r) {
    f(mx_check(gates[r], F, D));
    f(mx_check(ups[r], F, D));
    f(mx_check(acts[r], T, F));
    mx_ranges(in, gates[r], F, D);
    mx_ranges(in, ups[r], F, D);
    mx_ranges(o, acts[r], T, F);
  }
  f(too_many(T, plan.tiles(F) * nranks), RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, count, dt, 0, f.st);
  if (clash(in, o)) return done(call, nranks, count, dt, 0, RRA_ERR_ALIAS);
  if (count == 0) return done(call, nranks, 0, dt, 0, RRA_SUCCESS);
  if (!device_status()) return done(call, nranks, count, dt, 0, RRA_ERR_NOT_INITIALIZED);
  Mx4Args args;
  Mx4Args* const p = &args;
  start(p, T);
  one_segment(p, D);
  p->act = act;
  bool ok = map_mx(&p->x[0], &p->xs[0], *x, T, D, plan.x_box, 1);
  for (int r = 0; r < nranks && ok; ++r) {
    ok = map_mx(&p->w[2 * r], &p->ws[2 * r], gates[r], F, D, 128, plan.w_bands) &&
         map_mx(&p->w[2 * r + 1], &p->ws[2 * r + 1], ups[r], F, D, 128, plan.w_bands);
    Mx4Group& g = p->group[p->ngroups++];
    g.tile0 = p->tiles;
    g.tiles = (int)plan.tiles(F);
    g.rows = (int)F;
    g.w = 2 * r;
    g.out = acts[r].codes;
    g.out_scales = static_cast<uint8_t*>(acts[r].scales);
    g.across = (int)mx_across(F);
    g.ld = (long long)mx_row_bytes(F);
    p->tiles += g.tiles;
  }
  if (!ok) return done(call, nranks, count, dt, 0, RRA_ERR_CUDA);
  int grid = 0;
  const cudaError_t err = launch(p, plan, reinterpret_cast<cudaStream_t>(stream), &grid);
  return done(call, nranks, count, dt, grid, cuda_st(err));
}

rra_status_t rra_vocab_sample(const void* const* logits, const size_t* vocab, int nranks, size_t rows,
                              const float* uniform, const float* temperature, const int32_t* top_k,
                              const float* top_p, const float* min_p, int64_t* token, float* logprob,
                              rra_dtype_t dtype, rra_stream_t stream) {
  const char* call = "vocab_sample";
  First f;
  f(nranks > kMaxRanks, RRA_ERR_UNSUPPORTED);
  f(!logits || !vocab || nranks < 1 || !float_type(dtype) || (rows && (!uniform || !token)), RRA_ERR_INVALID_ARG);
  f(!aligned(uniform, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
        !aligned(min_p, 4) || !aligned(token, 8) || !aligned(logprob, 4),
    RRA_ERR_INVALID_ARG);
  f(bad_extent(rows), RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, 0, dtype, 0, f.st);
  const size_t e = size_of(dtype);
  SampleArgs a{};
  Ranges in;
  size_t V = 0;
  for (int r = 0; r < nranks; ++r) {
    f(vocab[r] > kSampleMaxVocab, RRA_ERR_UNSUPPORTED);
    if (f.st != RRA_SUCCESS) break;
    f((rows && vocab[r] && !logits[r]) || !aligned(logits[r], e), RRA_ERR_INVALID_ARG);
    in.push_back({logits[r], rows * vocab[r] * e});
    a.logits[r] = logits[r];
    V += vocab[r];
    a.first[r + 1] = (long long)V;
  }
  f(V > kSampleMaxVocab, RRA_ERR_UNSUPPORTED);
  if (f.st != RRA_SUCCESS) return done(call, nranks, rows * V, dtype, 0, f.st);
  in.push_back({uniform, rows * 4});
  in.push_back({temperature, temperature ? rows * 4 : 0});
  in.push_back({top_k, top_k ? rows * 4 : 0});
  in.push_back({top_p, top_p ? rows * 4 : 0});
  in.push_back({min_p, min_p ? rows * 4 : 0});
  if (clash(in, {{token, rows * 8}, {logprob, logprob ? rows * 4 : 0}}))
    return done(call, nranks, rows * V, dtype, 0, RRA_ERR_ALIAS);
  if (rows == 0) return done(call, nranks, 0, dtype, 0, RRA_SUCCESS);
  a.n = nranks;
  a.rows = rows;
  a.uniform = uniform;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.token = token;
  a.logprob = logprob;
  int grid = 0;
  const cudaError_t err = launch_vocab_sample(dtype, a, reinterpret_cast<cudaStream_t>(stream), &grid);
  return done(call, nranks, rows * V, dtype, grid, cuda_st(err));
}

}  // extern "C"
