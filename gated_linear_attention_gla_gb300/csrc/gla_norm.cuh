// gla_norm.cuh -- what the forward and backward kernels of the norms between blocks share:
// the threads that own a row and their sums.
#pragma once

#include "gla_ssm.cuh"

namespace gla {
namespace norm {

constexpr int kV = 8;           // channels a thread and vector
constexpr int kRedFloats = 2 * 2 * 32;  // two buffers of up to 32 warps' pairs of sums, per group

// Threads of a row, vectors of each, rows of a block.
struct Shape {
  int tpr, k, groups;
};

// The threads that own one row: `tpr` of them (whole warps), `count` groups a block.
struct Group {
  int index, count, lane, tpr;
  float* red;
  mutable int turn = 0;
  __device__ Group(int tpr_, float* shared)
      : index(threadIdx.x / tpr_), count(blockDim.x / tpr_), lane(threadIdx.x % tpr_), tpr(tpr_),
        red(shared + (threadIdx.x / tpr_) * kRedFloats) {}
  __device__ __forceinline__ int column(int k) const { return (k * tpr + lane) * kV; }

  // Sums over the group's threads, the same bits in each of them.  The two buffers
  // take turns: a thread writes one again only after a barrier behind its last reads.
  __device__ __forceinline__ float2 sum(float2 v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (tpr == 32) return v;
    float2* buf = reinterpret_cast<float2*>(red) + turn * 32;
    turn ^= 1;
    if ((lane & 31) == 0) buf[lane >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(tpr) : "memory");
    v = buf[0];
    for (int w = 1; w < tpr / 32; ++w) {
      v.x += buf[w].x;
      v.y += buf[w].y;
    }
    return v;
  }
  __device__ __forceinline__ float sum(float v) const { return sum(make_float2(v, 0.f)).x; }
};

// body(k, column) for the thread's vectors inside the row; zeros in x elsewhere.
template <int K, typename F>
__device__ __forceinline__ void each(const Group& g, int D, F body, float (&x)[K][kV]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = g.column(k);
    if (c < D) {
      body(k, c);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) x[k][j] = 0.f;
    }
  }
}

template <typename T> __device__ __forceinline__ void load_f32(const T* p, float (&x)[kV]) {
  unpack_as<T, kV>(load_raw<T, kV>(p), x);
}
__device__ __forceinline__ void load_vec(const float* p, float (&x)[kV]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Centres the row (layer norm) and returns 1 / sqrt(mean of squares + eps).
template <int K>
__device__ __forceinline__ float normalise(const Group& g, const NormArgs& a, float (&x)[K][kV]) {
  if (a.layer) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < kV; ++j) m += x[k][j];
    m = g.sum(m) * a.inv_d;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (g.column(k) < a.D)
#pragma unroll
        for (int j = 0; j < kV; ++j) x[k][j] -= m;
  }
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < kV; ++j) q = fmaf(x[k][j], x[k][j], q);
  return 1.f / sqrtf(g.sum(q) * a.inv_d + a.eps);
}

static_assert(kNormMaxD == 512 * 2 * kV, "the widest shape below");

// The fewest threads that hold a row with one or two vectors each.
inline Shape fwd_shape(int D) {
  const int vecs = (D + kV - 1) / kV;
  if (vecs <= 32) return {32, 1, 8};
  if (vecs <= 64) return {32, 2, 8};
  if (vecs <= 128) return {64, 2, 4};
  if (vecs <= 256) return {128, 2, 2};
  if (vecs <= 512) return {256, 2, 1};
  return {512, 2, 1};
}
inline Shape bwd_shape(int D) {
  const int vecs = (D + kV - 1) / kV;
  if (vecs <= 32) return {32, 1, 8};
  if (vecs <= 64) return {64, 1, 4};
  if (vecs <= 128) return {128, 1, 2};
  if (vecs <= 256) return {256, 1, 1};
  if (vecs <= 512) return {512, 1, 1};
  return {512, 2, 1};
}

}  // namespace norm
}  // namespace gla
