// gla_norm.cuh -- what the forward and backward kernels of the norms between blocks share:
// the threads that own a row, their sums and their rows in shared memory.
#pragma once

#include "gla_ssm.cuh"

namespace gla {
namespace norm {

constexpr int kV = 8;             // channels a thread and vector
constexpr int kMaxThreads = 512;  // of a row
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kRedFloats = 2 * 4 * kMaxWarps;  // two buffers of up to four sums of every warp, per group
static_assert(kNormMaxD == kMaxThreads * 2 * kV, "two vectors a thread at most");

// Threads of a row (whole warps), vectors of each, rows of a block.
struct Shape {
  int tpr, k, groups;
};
// The fewest threads that hold a row with one vector each, or with two above 4096 channels; 256
// threads a block at least.  With two vectors nothing is read ahead, the parameters are read for every row,
// and an SM has one block of 288 to 512 threads: rows of 67 MB a tensor (bf16, RMS, gate and scale) take 57 us
// at 2048 channels, 64 at 4096, 205 at 4104, 170 at 5120, 123 at 8192; gradients of half of them
// 55, 63, 195, 163 and 124.
inline Shape shape_of(int D) {
  const int vecs = (D + kV - 1) / kV, k = vecs <= kMaxThreads ? 1 : 2;
  const int tpr = ((vecs + k - 1) / k + 31) / 32 * 32;
  return {tpr, k, tpr >= 256 ? 1 : 256 / tpr};
}

// The threads that own a row (or a few rows at a time): `tpr` of them, `count` groups a block.
struct Group {
  int index, count, lane, tpr;
  float* red;
  mutable int turn = 0;
  __device__ Group(int tpr_, float* shared)
      : index(threadIdx.x / tpr_), count(blockDim.x / tpr_), lane(threadIdx.x % tpr_), tpr(tpr_),
        red(shared + (threadIdx.x / tpr_) * kRedFloats) {
    for (int i = lane; i < kRedFloats; i += tpr) red[i] = 0.f;  // (of warps that are not there)
    __syncthreads();
  }
  __device__ __forceinline__ int column(int k) const { return (k * tpr + lane) * kV; }

  // N sums (1, 2 or 4) over the group's threads, the same bits in each of them.  Inside a
  // warp the lanes' halves hand each other the sums they give up, so that two sums
  // cost the shuffles of one and four cost one more.  The two buffers take turns: a
  // thread writes one again only after a barrier behind its last reads.
  template <int N> __device__ __forceinline__ void sum(float (&v)[N]) const {
    static_assert(N == 1 || N == 2 || N == 4, "sums at a time");
    const int l = lane & 31;
    float x;
    if constexpr (N == 1) {
      x = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
    } else {
      const bool up = l & 16;
      float w[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        w[i] = (up ? v[N / 2 + i] : v[i]) +
               __shfl_xor_sync(0xffffffffu, up ? v[i] : v[N / 2 + i], 16);
      if constexpr (N == 2) {
        x = w[0] + __shfl_xor_sync(0xffffffffu, w[0], 8);
      } else {
        const bool second = l & 8;
        x = (second ? w[1] : w[0]) + __shfl_xor_sync(0xffffffffu, second ? w[0] : w[1], 8);
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    // sum i is in the lanes from i 32 / N on
    if (tpr == 32) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = N == 1 ? x : __shfl_sync(0xffffffffu, x, i * (32 / N));
      return;
    }
    float* buf = red + turn * 4 * kMaxWarps;
    turn ^= 1;
    if (l % (32 / N) == 0) buf[l / (32 / N) * kMaxWarps + (lane >> 5)] = x;
    asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(tpr) : "memory");
    if (tpr <= 128) gather<1>(buf, v);
    else if (tpr <= 256) gather<2>(buf, v);
    else gather<4>(buf, v);
  }

 private:
  template <int Q, int N>
  static __device__ __forceinline__ void gather(const float* buf, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      f32x2 t = both(0.f);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float4 x = reinterpret_cast<const float4*>(buf + i * kMaxWarps)[q];
        const f32x2 y = add2(make_float2(x.x, x.y), make_float2(x.z, x.w));
        t = q ? add2(t, y) : y;
      }
      v[i] = t.x + t.y;
    }
  }
};

// A thread's vector, as pairs: one instruction works on two channels.
struct Vec {
  f32x2 v[kV / 2];
};
__device__ __forceinline__ Vec vec_of(float x) {
  Vec r;
#pragma unroll
  for (int j = 0; j < kV / 2; ++j) r.v[j] = both(x);
  return r;
}
__device__ __forceinline__ Vec load_vec(const float* p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  Vec r;
  r.v[0] = make_float2(a.x, a.y); r.v[1] = make_float2(a.z, a.w);
  r.v[2] = make_float2(b.x, b.y); r.v[3] = make_float2(b.z, b.w);
  return r;
}
template <typename T> __device__ __forceinline__ void store_vec(T* p, const Vec& x) {
  float t[kV];
#pragma unroll
  for (int j = 0; j < kV / 2; ++j) unpack2(x.v[j], &t[2 * j], &t[2 * j + 1]);
  store_raw<T, kV>(p, pack_as<T, kV>(t));
}
#define GLA_PAIRS for (int j = 0; j < kV / 2; ++j)
// A parameter at the thread's columns: HELD over the rows, or loaded where it is used (where
// registers would not do: of two vectors a thread, of some in the backward kernel).
template <int K, bool HELD = K == 1> struct Param {
  Vec v;
  const float* p;
  float none;
  __device__ __forceinline__ void init(const Group& g, int D, const float* from, float otherwise) {
    p = from;
    none = otherwise;
    if constexpr (HELD) v = from && g.column(0) < D ? load_vec(from + g.column(0)) : vec_of(otherwise);
  }
  __device__ __forceinline__ Vec at(int column) const {
    if constexpr (HELD) return v;
    else return p ? load_vec(p + column) : vec_of(none);
  }
};

// A thread's vectors of the next rows in shared memory: its own copies, its own reads, no
// barrier.  Sixteen-byte pieces of all threads lie side by side, `per` a row.  With two
// vectors a thread (whose rows would not fit) the reads go to memory themselves.
constexpr int kMaxStages = 3;
__device__ __forceinline__ void cp_async16_or_0(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
template <typename T> constexpr int kPieces = kV * (int)sizeof(T) / 16;  // of a vector
template <int K> struct Ring {
  unsigned char* at;  // the thread's piece 0 of stage 0
  int hop;            // bytes between pieces
  int per, pieces, stages, stage = 0;  // pieces of a row, of a stage (which is R rows)
  __device__ Ring(void* shared, int R, int per_, int stages_)
      : at((unsigned char*)shared + threadIdx.x * 16), hop(blockDim.x * 16), per(per_),
        pieces(R * per_), stages(stages_) {}
  template <typename T>
  __device__ __forceinline__ void copy(int slot, int row, int first, const T* from) const {
#pragma unroll
    for (int i = 0; i < kPieces<T>; ++i)
      cp_async16(at + (slot * pieces + row * per + first + i) * hop,
                 (const unsigned char*)from + 16 * i);
  }
  // The same, or zeros, so that the reads need not ask (gradients of 8192 x 2048 82 -> 78 us; the
  // forward, whose time is its memory's, loses by it: 85 -> 91 us).
  template <typename T>
  __device__ __forceinline__ void copy_or_0(int slot, int row, int first, const T* from,
                                            bool on) const {
#pragma unroll
    for (int i = 0; i < kPieces<T>; ++i)
      cp_async16_or_0(at + (slot * pieces + row * per + first + i) * hop,
                      (const unsigned char*)from + 16 * i, on);
  }
  // The slot of the rows that are stages - 1 turns ahead.
  __device__ __forceinline__ int ahead() const { return stage == 0 ? stages - 1 : stage - 1; }
  __device__ __forceinline__ void next() { stage = stage == stages - 1 ? 0 : stage + 1; }
  // The current rows' copies have landed (of one group a turn).
  __device__ __forceinline__ void wait() const {
    if (stages == 3) cp_wait<2>();
    else if (stages == 2) cp_wait<1>();
    else cp_wait<0>();
  }
  // A vector of a current row: piece `first` on, or from memory.
  template <typename T>
  __device__ __forceinline__ Vec read(int row, int first, const T* from) const {
    Raw<T, kV> r;
    if constexpr (K == 1) {
#pragma unroll
      for (int i = 0; i < kPieces<T>; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(at + (stage * pieces + row * per + first + i) * hop);
        r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
      }
    } else {
      r = load_raw<T, kV>(from);
    }
    Vec x;
    unpack_pairs<T, kV>(r, x.v);
    return x;
  }
};
// Stages that fit beside `other` bytes, for `blocks` blocks an SM.
inline int ring_stages(int pieces, int threads, int other, int blocks) {
  const int room = 227 * 1024 / blocks - 1024 - other, n = room / (pieces * 16 * threads);
  return n < 1 ? 1 : n > kMaxStages ? kMaxStages : n;
}

// Centres R rows (layer norm) and leaves 1 / sqrt(mean of squares + eps) of each in r; 0
// for a row behind the last (of zeros), so that it adds nothing to sums over rows.  KIND: which
// of the norms, where the caller knows.
// Layer norm takes the sums of x and x^2 in one exchange, which loses (mean^2 / variance) of the sums'
// rounding to cancellation; rows whose mean is over half a deviation take the squares of the
// centred values in a second one, so that the variance is never off by much more than those would be (2048
// values: 2e-7 of it; up to four deviations in one exchange it would be 4e-6).  16384 x 2048, the norm alone,
// means of 0.4 deviations 30.8 us, of 0.6 37.0; gradients 61.4 and 75.8.
enum Kind { kRms, kEither };
__device__ __forceinline__ bool far_mean(float mean, float var) { return !(4.f * mean * mean <= var); }
template <int K, int R, int KIND = kEither>
__device__ __forceinline__ void normalise(const Group& g, const NormArgs& a, Vec (&x)[R][K],
                                          float (&r)[R], int rows) {
  auto squares = [&](int i) {
    f32x2 q = both(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      GLA_PAIRS q = fma2(x[i][k].v[j], x[i][k].v[j], q);
    return q.x + q.y;
  };
  const bool layer = KIND != kRms && a.layer;
  bool far = !layer;  // the squares are (again) to be taken
  if (layer) {
    float m[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      f32x2 t = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        GLA_PAIRS t = add2(t, x[i][k].v[j]);
      m[2 * i] = t.x + t.y;
      m[2 * i + 1] = squares(i);
    }
    g.sum(m);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float mean = m[2 * i] * a.inv_d, var = fmaf(-mean, mean, m[2 * i + 1] * a.inv_d);
      far |= far_mean(mean, var) && i < rows;
      r[i] = var;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (g.column(k) < a.D)
#pragma unroll
          GLA_PAIRS x[i][k].v[j] = add2(x[i][k].v[j], both(-mean));
    }
  }
  if (far) {  // (the same in all of the group's threads)
#pragma unroll
    for (int i = 0; i < R; ++i) r[i] = squares(i);
    g.sum(r);
#pragma unroll
    for (int i = 0; i < R; ++i) r[i] *= a.inv_d;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) r[i] = i < rows ? rsqrtf(r[i] + a.eps) : 0.f;
}

}  // namespace norm
}  // namespace gla
