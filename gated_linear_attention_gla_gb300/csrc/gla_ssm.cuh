// gla_ssm.cuh -- device helpers shared by the causal-convolution and
// selective-scan kernels: short vectors, sequence lookup by packed row, and
// the activations.
#pragma once

#include "gla_internal.cuh"

namespace gla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLo = 1.9259629891e-8f;  // log2(e) - kLog2e
constexpr float kLn2 = 0.6931471805599453f;

// 2^x by the hardware's approximation (flushes subnormal results to zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x / (1 + e^-x)
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + ex2(-kLog2e * x)); }
__device__ __forceinline__ float sigmoid(float x) {
  return __fdividef(1.f, 1.f + ex2(-kLog2e * x));
}

// e^-|x| with a relative error of a few 2^-24 (|x| up to 100; beyond that it
// is zero in fp32 anyway): the product with log2(e) is split, and what its
// rounding loses multiplies the result.
__device__ __forceinline__ float exp_neg_abs(float x) {
  const float m = -fminf(fabsf(x), 100.f);
  const float t = m * kLog2e;
  const float r = fmaf(m, kLog2e, -t) + m * kLog2eLo;
  const float e = ex2(t);
  return fmaf(e, r * kLn2, e);
}

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x| in (0, 1].  log1p(e) =
// 2 atanh(s) with s = e / (2 + e) <= 1/3: the series 2 s (1 + s^2/3 + s^4/5 +
// ...) up to s^12/13 leaves a relative remainder below s^14/15 < 2e-8, and
// keeps the relative accuracy for the small values (1e-4 .. 1e-1) that step
// sizes have.  *sig receives 1 / (1 + e^-x), its derivative.  A NaN stays one.
__device__ __forceinline__ float softplus(float x) {
  const float e = exp_neg_abs(x);
  const float s = __fdividef(e, 2.f + e), z = s * s;
  float p = 1.f / 13;
  p = fmaf(p, z, 1.f / 11);
  p = fmaf(p, z, 1.f / 9);
  p = fmaf(p, z, 1.f / 7);
  p = fmaf(p, z, 1.f / 5);
  p = fmaf(p, z, 1.f / 3);
  p = fmaf(p, z, 1.f);
  return fmaf(2.f * s, p, x < 0.f ? 0.f : x);
}

// V consecutive elements as they lie in memory (V * sizeof(T) = 4, 8 or 16 bytes).
template <int BYTES> struct RawOf;
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
template <typename T, int V> using Raw = typename RawOf<V * (int)sizeof(T)>::type;

template <int V> __device__ __forceinline__ void unpack(const Raw<float, V>& r, float (&x)[V],
                                                        float) {
  const float* p = reinterpret_cast<const float*>(&r);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = p[i];
}
template <int V> __device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, V>& r,
                                                        float (&x)[V], __nv_bfloat16) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    x[2 * i] = __uint_as_float(p[i] << 16);
    x[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
  }
}
template <typename T, int V> __device__ __forceinline__ void unpack_as(const Raw<T, V>& r,
                                                                       float (&x)[V]) {
  unpack<V>(r, x, T());
}
template <typename T, int V> __device__ __forceinline__ Raw<T, V> pack_as(const float (&x)[V]) {
  Raw<T, V> r;
  if constexpr (sizeof(T) == 4) {
    float* p = reinterpret_cast<float*>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = x[i];
  } else {
    __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  }
  return r;
}
template <typename T, int V> __device__ __forceinline__ Raw<T, V> zero_raw() {
  Raw<T, V> r;
  uint32_t* p = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < V * (int)sizeof(T) / 4; ++i) p[i] = 0u;
  return r;
}

// Bounds [a, b) of sequence s in packed rows (dense batches: s * T ..).
__device__ __forceinline__ void seq_rows(const int32_t* cu, int s, int T, long long* a,
                                         long long* b) {
  if (cu == nullptr) {
    *a = (long long)s * T;
    *b = *a + T;
  } else {
    *a = __ldg(cu + s);
    *b = __ldg(cu + s + 1);
  }
}

// The sequence that holds packed row r: the first s with cu[s + 1] > r.  For
// any contents of cu the answer lies in [0, B).
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int B, int T, long long r) {
  if (cu == nullptr) return (int)(r / T);
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid + 1) > r) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

}  // namespace gla
