// serve_host.h -- what the host planning of the serving-step operators
// (rra_serve.cpp) and their kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "rra_internal.h"
#include "tc_host.h"

namespace rra {

// kernels_mx4.cu
cudaError_t launch_mx4_quantize(int dt, bool vec, const void* x, void* codes, void* scales, size_t rows, size_t cols,
                                cudaStream_t s);
cudaError_t launch_mx4_restore(int dt, bool vec, const void* codes, const void* scales, void* out, size_t rows,
                               size_t cols, cudaStream_t s);
cudaError_t launch_norm_mx4(int n, int dt, bool vec, const void* const* in, const void* residual, void* residual_out,
                            const void* gamma, size_t rows, size_t hidden, float eps, void* codes, void* scales,
                            cudaStream_t s);

// ---------------------------------------------------------------------------
// products of MX4 matrices (kernels_mx4_product.cu, kernels_mx4_few.cu)
// ---------------------------------------------------------------------------
constexpr int kMxKTile = 256;  // columns per stage: 128 bytes of codes, two tiles of scales

// One rank's output: rows of its weights are columns of `out`.
struct Mx4Group {
  int tile0;   // first weight tile of the group
  int tiles;   // weight tiles
  int rows;    // weight rows
  int w;       // first of its tensor maps (gated: gate, then up)
  int vec;     // rows of out start on 16 bytes
  int across;  // gated: scale tiles of a row band of the output
  void* out;   // tokens x rows, or the codes of a gated block's activations
  uint8_t* out_scales;
  long long ld;  // elements (codes: bytes) between rows of out
};

struct Mx4Args {
  CUtensorMap x[kMaxRanks], xs[kMaxRanks];          // codes and scales of the activations, one per K segment
  CUtensorMap w[2 * kMaxRanks], ws[2 * kMaxRanks];  // of the weights: per group, or per K segment
  Mx4Group group[kMaxRanks];
  int seg_k0[kMaxRanks];  // first K tile of each segment
  int ngroups, nsegs;
  int tiles;    // weight tiles of all groups
  int kblocks;  // K tiles of all segments
  int tokens;
  int mt;       // token tiles
  int act;
  int f32;      // out is float32
  int split;    // few tokens: CTAs of a cluster that share a tile's K axis
  int stages;   // few tokens: stages of the ring
  DevStatus* status;
};

// Codes: rows of `row_bytes` bytes in boxes of 128 bytes x box_rows; scales:
// bands of `across` tiles in boxes of two tiles x box_bands.
bool mx4_map_codes(CUtensorMap* m, const void* base, size_t row_bytes, size_t rows, int box_rows);
bool mx4_map_scales(CUtensorMap* m, const void* base, size_t across, size_t bands, int box_bands);

// Many tokens: tiles of 256 tokens x 256 weight rows (gated: 128 of the gate's
// and the same 128 of the up projection's).
cudaError_t launch_mx4_product(const Mx4Args& p, bool gated, cudaStream_t s, int* grid);
// Few: tiles of 128 weight rows x all tokens, for calls of
// mx4_few_most(weight rows, gated) tokens at most.
size_t mx4_few_most(size_t rows, bool gated);
int mx4_few_tile(size_t tokens);  // columns of a tile
// Picks p.split and p.stages.
cudaError_t launch_mx4_few(Mx4Args& p, bool gated, cudaStream_t s, int* grid);

// kernels_vocab_sample.cu
constexpr size_t kSampleMaxVocab = 360 * 1024;  // a row's logits lie in the shared memory of 8 CTAs
struct SampleArgs {
  const void* logits[kMaxRanks];
  long long first[kMaxRanks + 1];  // index of each shard's first column
  int n;
  size_t rows;
  const float* uniform;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int64_t* token;
  float* logprob;
};
cudaError_t launch_vocab_sample(int dt, const SampleArgs& a, cudaStream_t s, int* grid);

}  // namespace rra
