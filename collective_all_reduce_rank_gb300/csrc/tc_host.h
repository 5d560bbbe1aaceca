// tc_host.h -- what the host planning of the training operators and their
// tensor-core kernels share: argument structs, tensor maps, launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "rra_internal.h"

namespace rra {

constexpr int kTcMaxGroups = 2 * kMaxRanks;
constexpr int kTcKBlock = 64;              // K elements per stage (128 bytes)
constexpr int kTcBand = 8;  // tile rows per band of the tile walk

// One output of a launch: an M x N product tiled 256 x 256.  `a` and `b`
// index the tensor maps (unused when the launch walks K segments).
struct TcGroup {
  int a, b;
  int tile0;   // first tile of the group
  int mt, nt;  // tiles
  int M, N;    // extents of the output (rows and columns stored)
  int m0, n0;  // where the group starts along A's and B's M / N axes
  void* out;
  void* out2;
  const void* in;
  long long ld;     // elements between rows of out (and out2)
  long long ld_in;  // elements between rows of in
  int vec;          // rows of out (and in) start on 16 bytes
  long long col0;   // global column of this group's column 0
  int part0;        // column tiles of the groups before this one
};

// What a CTA stages of A per K block.  Few tokens leave most of A's 128 rows
// out of range: only the rows there are are loaded (the products read what
// lies behind them, into rows of C that nobody reads), and the ring gets as
// many stages as fit, so that more of the weights, which then bound the call,
// are on their way (hidden 5120, 131072 columns, 17 tokens: 224 us with 6
// stages, 213 with 10; 17 tokens through 8 x 1728 gated columns 60 and 56).
struct TcShape {
  int a_rows = 128;  // rows of A loaded per CTA
  int a_ctas = 2;    // CTAs of the pair that have rows of A
  int stages = 6;
};

// Rank-one additions to the loss's gradients, in float32 before the result
// is rounded: column[t] is the target of token t (-1: none), lo[t] a factor.
// kind 1 (dx): row t += lo[t] row column[t] of the shards w; kind 2 (dW, the
// group's first row being column col0): row column[t] += lo[t] row t of w[0],
// the tokens taken from an index by target: those of a shard's 32 rows from
// 32 b on are token[start[k]], ..., token[start[k + 1] - 1] with targets
// sorted[...], k = b plus the blocks of the shards before (the group's first
// block is part0).
struct TcFix {
  int kind = 0;
  const int* column;
  const float* lo;
  const int* start;
  const int* token;
  const int* sorted;
  const void* w[kMaxRanks];
  long long first[kMaxRanks + 1];
  long long ld;  // elements between rows, which hold whole 16-byte units
};

struct TcArgs {
  CUtensorMap a[kTcMaxGroups];
  CUtensorMap b[kTcMaxGroups];
  TcGroup group[kTcMaxGroups];
  int seg_k0[kTcMaxGroups];  // first K block of each segment
  int ngroups, nsegs;
  int tiles;    // tiles of all groups
  int full;     // the first `full` tiles of the walk take the whole K axis,
  int splits;   // the others one of `splits` parts of it at a time (tc_units)
  int kblocks;  // K blocks of 64 over all segments
  int rest_k;   // two segments of the same maps, A's second one from row rest_k on (0: not so)
  TcShape shape;
  int pair_b;   // CTA c of a pair takes map b + c (gate and up weights), 128 columns per tile each
  // epilogue operands
  float* slots;    // split tiles: 256 x 256 float32 per part, part v of tile full + v / splits
  int accumulate;  // add to the float32 outputs
  int act;
  const long long* targets;
  long long ignore_index;
  const float4* rows;  // dl: what loss_rows_kernel left per row
  int rest_row;        // dl, dg and du: rows from here on take what bfloat16 leaves of the others (0: not kept)
  TcFix fix;
  float2* part;      // [column part][part_ld] running maximum and sum
  long long part_ld;
  float* hit;        // logit of the row's target
  DevStatus* status;
};

// Clusters of two CTAs to launch for `tiles` tiles: one per SM pair, at
// most the SM budget.
int tc_clusters(int tiles);

// Tensor maps over a dense matrix of bfloat16: `inner` contiguous elements,
// `rows` rows, `ld` elements from row to row (a multiple of 8), 16-byte
// aligned base.  K-major boxes are 64 x 128 (K x rows of M or N), MN-major
// boxes 64 x 64 (M or N x rows of K).  `box`: rows of a K-major box.  False
// if the driver refuses.
bool tc_map(CUtensorMap* m, const void* base, size_t inner, size_t rows, size_t ld, bool mn_major, int box);

// Products (kernels_vocab_loss.cu, kernels_gated_ffn.cu, kernels_tc_store.cu)
cudaError_t launch_tc_lse(const TcArgs& p, cudaStream_t s, int* grid);        // K-major x K-major
cudaError_t launch_tc_dlogits(const TcArgs& p, cudaStream_t s, int* grid);    // K-major x K-major
cudaError_t launch_tc_gate(const TcArgs& p, cudaStream_t s, int* grid);       // K-major x K-major
cudaError_t launch_tc_gate_back(const TcArgs& p, cudaStream_t s, int* grid);  // K-major x K-major
// out = A B for A K-major, B MN-major (the gradient of the input): bfloat16
// rows, or float32 rows (added to when p.accumulate); split tiles go to
// p.slots either way.
cudaError_t launch_tc_input_grad(const TcArgs& p, bool f32, cudaStream_t s, int* grid);
// out = A^T B, both MN-major (the gradient of the weights): bfloat16 rows.
cudaError_t launch_tc_weight_grad(const TcArgs& p, cudaStream_t s, int* grid);

// Few tokens (kernels_skinny.cu): at most 16 (rra_train.cpp says when).
struct SkinnyArgs {
  const void* x;
  const void* w[2 * kMaxRanks];  // gate and up shards in turn, or vocabulary shards
  void* out[kMaxRanks];
  int tokens, hidden, width;
  int units;
  int unit0[kMaxRanks + 1];  // loss: first unit of each shard
  long long rows[kMaxRanks], col0[kMaxRanks];
  const long long* targets;
  long long ignore_index;
  float2* part;  // [grid][tokens]
  float* hit;
};
int skinny_most(long long units);  // CTAs without an SM budget: what a workspace holds parts for
int skinny_grid(long long units);
// Units of a shard: 8 gated columns or 16 vocabulary rows each (vec: rows of
// whole 16-byte units), counted in whole blocks of 64 or 128 otherwise.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int sk_gate_units(int width, bool vec) { return vec ? (width + 7) / 8 : (width + 63) / 64 * 8; }
inline long long sk_loss_units(long long rows, bool vec) { return vec ? (rows + 15) / 16 : (rows + 127) / 128 * 8; }
cudaError_t launch_skinny_gate(const SkinnyArgs& a, int act, cudaStream_t s, int* grid);
cudaError_t launch_skinny_lse(const SkinnyArgs& a, cudaStream_t s, int* grid);

// Row-wise helpers
// part: [parts][rows] running maximum and sum of each column part; hit: the
// product's logit of each row's target.
cudaError_t launch_loss_join(const float2* part, int parts, const float* hit, const long long* targets,
                             long long ignore_index, const void* x, const void* const* w, const size_t* vocab, int n,
                             size_t hidden, int rows, float* loss, float* lse, cudaStream_t s);
// dx from what the products of its one group of tiles left: tiles that took
// the whole K axis are in `acc` (float32 rows of ld; null: already in out),
// the others the sum of their parts in `slots`.  rest: rows that far down are
// added to the first ones (the second halves of A's entries, in the same tile).
struct JoinTiles {
  const float* acc;
  const float* slots;
  void* out;
  int ld, rows, cols, mt, nt, full, splits;
  TcFix fix;  // kind 1 or none
  int rest = 0;
};
cudaError_t launch_join_tiles(const JoinTiles& j, cudaStream_t s);
// Units of work of a launch: whole tiles, then parts of the others.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int tc_units(const TcArgs& p) { return p.full + (p.tiles - p.full) * p.splits; }
// Per row of the loss's backward pass: rows[t] = {lse / log 2, the target's
// entry of dl in bfloat16, 1 or 0 (no gradient), grad}; TcFix's arrays.
cudaError_t launch_loss_rows(const void* x, const void* const* w, const size_t* vocab, int n, size_t hidden, int tokens,
                             const long long* targets, long long ignore_index, const float* lse, const float* grad,
                             float4* rows, int* column, float* lo, int* start, int* token, int* sorted,
                             cudaStream_t s);

// Rows of `cols` elements of each src to rows of 8 * units elements of dst.
struct PadArgs {
  const void* src[kTcMaxGroups + 1];
  void* dst[kTcMaxGroups + 1];
  long long first[kTcMaxGroups + 2];  // first 16-byte unit of each matrix
  long long cols;
  int units;  // 16-byte units of a destination row
  int n;
};
cudaError_t launch_pad_rows(const PadArgs& a, cudaStream_t s);

// Training-side norm kernels (kernels_norm8.cu)
constexpr int kCkptBlock = 128;
cudaError_t launch_norm_save8(int n, int dt, bool vec, const void* const* in, void* const* out, const void* gamma,
                              size_t rows, size_t hidden, float eps, void* codes, void* scales, float* rstd,
                              cudaStream_t s);
cudaError_t launch_norm_restore8(int dt, bool vec, const void* codes, const void* scales, const float* rstd,
                                 const void* gamma, void* out, size_t rows, size_t hidden, cudaStream_t s);
// CTAs of the backward kernel (each leaves one row of dgamma partials)
int norm_back8_ctas(size_t rows);
size_t norm_back8_pitch(size_t hidden);  // float32 per row of partials
cudaError_t launch_norm_back8(int n, int dt, bool vec, const void* const* grads, void* const* dxs,
                              const void* codes, const void* scales, const float* rstd, const void* gamma,
                              float* dgamma, float* part, size_t rows, size_t hidden, cudaStream_t s);

// Device status word of rra_init on the current device (null: not initialised).
DevStatus* device_status();
int device_sms();

}  // namespace rra
