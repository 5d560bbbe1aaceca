// abi_util.h -- argument checks that the C entry points of the training and
// serving operators share.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "rra.h"
#include "rra_internal.h"

namespace rra {

constexpr size_t kAlign = 256;

inline size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Range {
  const void* p;
  size_t bytes;
};

inline bool meet(const Range& a, const Range& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// A call's address ranges (no allocation, so nothing here can throw).
struct Ranges {
  Range r[8 + 6 * kMaxRanks];
  size_t n = 0;
  Ranges() = default;
  Ranges(std::initializer_list<Range> l) {
    for (const Range& x : l) push_back(x);
  }
  void push_back(const Range& x) { r[n++] = x; }
  size_t size() const { return n; }
  const Range& operator[](size_t i) const { return r[i]; }
};

// An output meets an input or another output; of the first `inplace` pairs,
// output i may be input i.
inline bool clash(const Ranges& in, const Ranges& out, int inplace = 0) {
  for (size_t i = 0; i < out.size(); ++i) {
    for (size_t j = i + 1; j < out.size(); ++j)
      if (meet(out[i], out[j])) return true;
    for (size_t j = 0; j < in.size(); ++j)
      if (meet(out[i], in[j]) && !(i == j && (int)i < inplace && out[i].p == in[j].p)) return true;
  }
  return false;
}

inline rra_status_t cuda_st(cudaError_t e) { return e == cudaSuccess ? RRA_SUCCESS : RRA_ERR_CUDA; }

// Ends a call: its record has the largest grid of its launches.
inline rra_status_t done(const char* call, int n, size_t count, int dt, int grid, rra_status_t st) {
  return record_call(call, RRA_ALGO_DIRECT, n, count, dt, std::max(grid, take_grid()), st);
}

}  // namespace rra
