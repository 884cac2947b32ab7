// gla_checks.cuh -- the argument checks shared by the entry points (host code).
#pragma once

#include <cstddef>
#include <cstdint>

#include "gla.h"
#include "gla_internal.cuh"

namespace gla {
namespace checks {

constexpr long long kMaxElems = 1ll << 40;  // per tensor; keeps index arithmetic exact
constexpr long long kMaxGrid = 0x7fffffffll;

inline bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// A byte range of a call's arguments.
struct Range {
  const void* p;
  size_t n;
};
inline bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// every output apart from every input and from the other outputs
template <int I, int O> bool disjoint(const Range (&in)[I], const Range (&out)[O]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (overlap(out[o], in[i])) return false;
    for (int o2 = o + 1; o2 < O; ++o2)
      if (overlap(out[o], out[o2])) return false;
  }
  return true;
}

// Bytes spanned by `rows` rows of `cols` elements, `stride` elements apart.
inline size_t span(long long rows, long long stride, long long cols, long long esz) {
  return rows > 0 ? (size_t)(((rows - 1) * stride + cols) * esz) : 0;
}

// More than kMaxElems elements (whose number need not fit 64 bits).
inline bool too_many(long long rows, long long stride) { return stride > 0 && rows > kMaxElems / stride; }

inline gla_status finish(cudaError_t e) { return static_cast<gla_status>(gla::cuda_result(e)); }

inline bool channels_ok(int D) { return D % 8 == 0 && D <= 1 << 24; }

// Rows, channel count and row strides shared by the entry points:
// stride rows must hold the columns and keep every row 16-byte aligned.
inline bool stride_bad(long long stride, int cols) { return stride < cols || stride > kMaxElems; }
inline bool stride_misaligned(long long stride, long long esz) { return stride * esz % 16 != 0; }

}  // namespace checks
}  // namespace gla
