// gla_norm.cuh -- what the forward and backward kernels of the norms between blocks share:
// the threads that own a row, their sums and their rows in shared memory.
#pragma once

#include "gla_ssm.cuh"

namespace gla {
namespace norm {

constexpr int kV = 8;             // channels a thread and vector
constexpr int kMaxThreads = 512;  // of a row
constexpr int kRedFloats = 2 * 2 * 32;  // two buffers of up to 32 warps' pairs of sums, per group
static_assert(kNormMaxD == kMaxThreads * 2 * kV, "two vectors a thread at most");

// Threads of a row (whole warps), vectors of each, rows of a block.
struct Shape {
  int tpr, k, groups;
};
// The fewest threads that hold a row with one vector each, or with two above 4096 channels; 256
// threads a block at least.
inline Shape shape_of(int D) {
  const int vecs = (D + kV - 1) / kV, k = vecs <= kMaxThreads ? 1 : 2;
  const int tpr = ((vecs + k - 1) / k + 31) / 32 * 32;
  return {tpr, k, tpr >= 256 ? 1 : 256 / tpr};
}

// The threads that own one row: `tpr` of them, `count` groups a block.
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
    for (int o = 16; o > 0; o >>= 1) v = add2(v, shfl_xor2(v, o));
    if (tpr == 32) return v;
    float2* buf = exchange();
    if ((lane & 31) == 0) buf[lane >> 5] = v;
    wait();
    v = buf[0];
    for (int w = 1; w < tpr / 32; ++w) v = add2(v, buf[w]);
    return v;
  }
  __device__ __forceinline__ float sum(float v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    float* buf = reinterpret_cast<float*>(exchange());
    if ((lane & 31) == 0) buf[lane >> 5] = v;
    wait();
    v = buf[0];
    for (int w = 1; w < tpr / 32; ++w) v += buf[w];
    return v;
  }

 private:
  __device__ __forceinline__ float2* exchange() const {
    float2* buf = reinterpret_cast<float2*>(red) + turn * 32;
    turn ^= 1;
    return buf;
  }
  __device__ __forceinline__ void wait() const {
    asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(tpr) : "memory");
  }
};

__device__ __forceinline__ void load_vec(const float* p, float (&x)[kV]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void fill(float (&x)[kV], float v) {
#pragma unroll
  for (int j = 0; j < kV; ++j) x[j] = v;
}
// A parameter at the thread's columns: held over the rows (one vector a thread), or loaded
// where it is used (two, whose registers would not do).
template <int K> struct Param {
  float v[K == 1 ? kV : 1];
  const float* p;
  float none;
  __device__ __forceinline__ void init(const Group& g, int D, const float* from, float otherwise) {
    p = from;
    none = otherwise;
    if constexpr (K == 1) {
      if (from && g.column(0) < D) load_vec(from + g.column(0), v);
      else fill(v, otherwise);
    }
  }
  __device__ __forceinline__ void at(int column, float (&x)[kV]) const {
    if constexpr (K == 1) {
#pragma unroll
      for (int j = 0; j < kV; ++j) x[j] = v[j];
    } else if (p) {
      load_vec(p + column, x);
    } else {
      fill(x, none);
    }
  }
};

// A thread's vectors of the next rows in shared memory: its own copies, its own reads, no
// barrier.  Sixteen-byte pieces of all threads lie side by side, `pieces` a row.  With two
// vectors a thread (whose rows would not fit) the reads go to memory themselves.
constexpr int kMaxStages = 3;
template <typename T> constexpr int kPieces = kV * (int)sizeof(T) / 16;  // of a vector
template <int K> struct Ring {
  unsigned char* at;  // the thread's piece 0 of stage 0
  int hop;            // bytes between pieces
  int pieces, stages, stage = 0;
  __device__ Ring(void* shared, int pieces_, int stages_)
      : at((unsigned char*)shared + threadIdx.x * 16), hop(blockDim.x * 16), pieces(pieces_),
        stages(stages_) {}
  template <typename T>
  __device__ __forceinline__ void copy(int slot, int first, const T* from) const {
#pragma unroll
    for (int i = 0; i < kPieces<T>; ++i)
      cp_async16(at + (slot * pieces + first + i) * hop, (const unsigned char*)from + 16 * i);
  }
  // The slot of the row that is stages - 1 rows ahead.
  __device__ __forceinline__ int ahead() const { return stage == 0 ? stages - 1 : stage - 1; }
  __device__ __forceinline__ void next() { stage = stage == stages - 1 ? 0 : stage + 1; }
  // The current row's copies have landed (of one group a row).
  __device__ __forceinline__ void wait() const {
    if (stages == 3) cp_wait<2>();
    else if (stages == 2) cp_wait<1>();
    else cp_wait<0>();
  }
  // A vector of the current row: piece `first` on, or from memory.
  template <typename T>
  __device__ __forceinline__ void read(int first, const T* from, float (&x)[kV]) const {
    Raw<T, kV> r;
    if constexpr (K == 1) {
#pragma unroll
      for (int i = 0; i < kPieces<T>; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(at + (stage * pieces + first + i) * hop);
        r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
      }
    } else {
      r = load_raw<T, kV>(from);
    }
    unpack_as<T, kV>(r, x);
  }
};
// Stages that fit beside `other` bytes, for `blocks` blocks an SM.
inline int ring_stages(int pieces, int threads, int other, int blocks) {
  const int room = 227 * 1024 / blocks - 1024 - other, n = room / (pieces * 16 * threads);
  return n < 1 ? 1 : n > kMaxStages ? kMaxStages : n;
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

}  // namespace norm
}  // namespace gla
