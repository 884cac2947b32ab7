// gla_ssm.cuh -- device helpers shared by the causal-convolution and
// selective-scan kernels: short vectors, sequence lookup by packed row, and
// the activations.
#pragma once

#include "gla_internal.cuh"

namespace gla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLo = 1.9259630e-8f;  // log2(e) - kLog2e
constexpr float kLn2 = 0.6931471805599453f;

// 2^x by the hardware's approximation (flushes subnormal results to zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x by the hardware's approximation (1 / inf = 0).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x / (1 + e^-x)
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// Two fp32 values in one register pair: one instruction works on both.  (Of the
// pair's type the compiler allocates pairs throughout; with 64-bit integers and
// inline instructions it moved every exponential's result into place first, ten
// instructions a token in the scan's recurrence.)
using f32x2 = float2;
__device__ __forceinline__ f32x2 pack2(float x, float y) { return make_float2(x, y); }
__device__ __forceinline__ void unpack2(f32x2 v, float* x, float* y) {
  *x = v.x;
  *y = v.y;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ f32x2 ex2x2(f32x2 v) { return make_float2(ex2(v.x), ex2(v.y)); }
__device__ __forceinline__ f32x2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ f32x2 shfl_xor2(f32x2 v, int lanes) {
  return make_float2(__shfl_xor_sync(0xffffffffu, v.x, lanes),
                     __shfl_xor_sync(0xffffffffu, v.y, lanes));
}

// e^-|x| of two values.  The rounding of the product with log2(e) costs up to
// |x| 2^-24 of the result; EXACT multiplies what it lost back in.
template <bool EXACT> __device__ __forceinline__ f32x2 exp_neg_abs2(f32x2 v) {
  const f32x2 m = make_float2(-fabsf(v.x), -fabsf(v.y));
  const f32x2 t = mul2(m, both(kLog2e));
  f32x2 e = ex2x2(t);
  if (EXACT) {
    // (beyond 2^-126 the result is zero, and infinite arguments must not give NaN)
    const f32x2 c = make_float2(fmaxf(m.x, -100.f), fmaxf(m.y, -100.f));
    const f32x2 lost = fma2(c, both(kLog2eLo),
                            fma2(c, both(kLog2e), mul2(c, both(-kLog2e))));
    e = fma2(e, mul2(lost, both(kLn2)), e);
  }
  return e;
}

// 2^t of two values, the decays of a token (t > 0 and decays above 1 where a step size
// or a is of the other sign).  The hardware's approximation is off by a part of
// 2^-23 and more to one side than to the other, which a state that lives for
// hundreds of tokens adds up; EXACT (fp32 rows) takes decays next to 1, |t| < 1/16,
// from the Taylor series (its rest: 1.3e-9), rounded once at the end.  777
// fp32 rows, 520 channels, 8 states, against 64 bits: gradient of dt_bias off by
// 1.3e-6 without, 2.7e-7 with; 4096 x 2048 x 16 fp32 prompt 60 -> 77 us.
template <bool EXACT> __device__ __forceinline__ f32x2 decay2(f32x2 t) {
  const f32x2 e = ex2x2(t);
  if (!EXACT) return e;
  // ln(2)^k / k!
  f32x2 p = fma2(both(9.6181291e-3f), t, both(5.5504109e-2f));
  p = fma2(p, t, both(0.24022651f));
  p = fma2(p, t, both(kLn2));
  p = fma2(p, t, both(1.f));
  return make_float2(fabsf(t.x) < 0.0625f ? p.x : e.x, fabsf(t.y) < 0.0625f ? p.y : e.y);
}

// log(1 + e^x) of two values = max(x, 0) + log1p(e), e = e^-|x| in (0, 1].
// log1p(e) = 2 atanh(s) with s = e / (2 + e) <= 1/3, and atanh(s) / s is a
// polynomial in s^2 <= 1/9: the degree-4 one below (fitted for the least
// relative error there) is off by 4e-9.  So the small step sizes (1e-4 ..
// 1e-1) keep their relative accuracy: below 1e-6 for |x| <= 12, 1e-7 on
// average, all but 2e-7 of it from the rounding that EXACT takes back (for fp32
// rows; in bf16 ones dt itself is known to 2^-9).  A NaN stays one.
template <bool EXACT> __device__ __forceinline__ f32x2 softplus2(f32x2 v) {
  const f32x2 e = exp_neg_abs2<EXACT>(v);
  const f32x2 d = add2(e, both(2.f));
  const f32x2 s = mul2(e, make_float2(rcp(d.x), rcp(d.y)));
  const f32x2 z = mul2(s, s);
  f32x2 p = fma2(both(0.14089167f), z, both(0.13980301f));
  p = fma2(p, z, both(0.20012455f));
  p = fma2(p, z, both(0.33333158f));
  p = fma2(p, z, both(1.f));
  // (x < 0 ? 0 : x keeps a NaN)
  return fma2(mul2(s, p), both(2.f), make_float2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y));
}
template <bool EXACT> __device__ __forceinline__ float softplus(float x) {
  return softplus2<EXACT>(both(x)).x;
}

// the sigmoids of two values
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
  const f32x2 d = add2(ex2x2(mul2(x, both(-kLog2e))), both(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}
// softplus' derivative, 1 / (1 + e^-x), as accurate as softplus2
template <bool EXACT> __device__ __forceinline__ f32x2 softplus_slope2(f32x2 x) {
  if (!EXACT) return sigmoid2(x);
  const f32x2 e = exp_neg_abs2<true>(x), d = add2(e, both(1.f));
  return mul2(make_float2(x.x < 0.f ? e.x : 1.f, x.y < 0.f ? e.y : 1.f),
              make_float2(rcp(d.x), rcp(d.y)));
}

// V consecutive elements as they lie in memory (4, 8, 16 or 32 bytes), as words.
template <int WORDS> struct alignas(WORDS >= 4 ? 16 : WORDS * 4) Words {
  uint32_t w[WORDS];
};
template <typename T, int V> using Raw = Words<V * (int)sizeof(T) / 4>;

template <int N> __device__ __forceinline__ Words<N> load_words(const void* p) {
  Words<N> r;
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = static_cast<const uint4*>(p)[i / 4];
      r.w[i] = v.x; r.w[i + 1] = v.y; r.w[i + 2] = v.z; r.w[i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = *static_cast<const uint2*>(p);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
    r.w[0] = *static_cast<const uint32_t*>(p);
  }
  return r;
}
template <int N> __device__ __forceinline__ void store_words(void* p, const Words<N>& r) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      static_cast<uint4*>(p)[i / 4] = make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]);
  } else if constexpr (N == 2) {
    *static_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
  } else {
    *static_cast<uint32_t*>(p) = r.w[0];
  }
}
template <typename T, int V> __device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
  return load_words<V * (int)sizeof(T) / 4>(p);
}
template <typename T, int V> __device__ __forceinline__ void store_raw(T* p, const Raw<T, V>& r) {
  store_words(p, r);
}

// the same as pairs: x[i] = elements 2 i, 2 i + 1
template <typename T, int V>
__device__ __forceinline__ void unpack_pairs(const Raw<T, V>& r, f32x2 (&x)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    if constexpr (sizeof(T) == 4)
      x[i] = pack2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    else
      x[i] = pack2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
  }
}
template <typename T, int V>
__device__ __forceinline__ void unpack_as(const Raw<T, V>& r, float (&x)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      x[2 * i] = __uint_as_float(r.w[i] << 16);
      x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  }
}
template <typename T, int V> __device__ __forceinline__ Raw<T, V> pack_as(const float (&x)[V]) {
  Raw<T, V> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)  // two conversions, round to nearest even; x[2 i] low
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  }
  return r;
}
template <typename T, int V> __device__ __forceinline__ Raw<T, V> zero_raw() {
  Raw<T, V> r;
#pragma unroll
  for (int i = 0; i < V * (int)sizeof(T) / 4; ++i) r.w[i] = 0u;
  return r;
}

// 16 bytes global -> shared without registers; a thread's copies form groups, and
// cp_wait<N> waits until at most its N newest groups are outstanding.
__device__ __forceinline__ void cp_async16(void* shared, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(shared))),
               "l"(global)
               : "memory");
}
// 8 or 16 bytes
template <int BYTES> __device__ __forceinline__ void cp_async(void* shared, const void* global) {
  static_assert(BYTES == 8 || BYTES == 16, "sizes of an asynchronous copy");
  if constexpr (BYTES == 16) {
    cp_async16(shared, global);
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(shared))),
                 "l"(global)
                 : "memory");
  }
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The filters [V][W] of V adjacent channels (16-byte aligned: V is a multiple of
// 4), as 16-byte loads: neighbouring lanes' filters lie V * W * 4 bytes apart, and every
// load instruction costs the cache a pass per lane, so few wide ones are cheap.
template <int W, int V>
__device__ __forceinline__ void load_filters(const float* weight, float (&w)[V][W]) {
#pragma unroll
  for (int i = 0; i < V * W / 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(weight) + i);
    w[(4 * i) / W][(4 * i) % W] = v.x;
    w[(4 * i + 1) / W][(4 * i + 1) % W] = v.y;
    w[(4 * i + 2) / W][(4 * i + 2) % W] = v.z;
    w[(4 * i + 3) / W][(4 * i + 3) % W] = v.w;
  }
}

// Bounds [a, b) of sequence s in packed rows (dense batches: s * T ..).  A negative
// offset, which is malformed, comes out above every row (as unsigned), so that a
// comparison with a row from above is enough to refuse it.
__device__ __forceinline__ void seq_rows(const int32_t* cu, int s, int T, long long* a,
                                         long long* b) {
  if (cu == nullptr) {
    *a = (long long)s * T;
    *b = *a + T;
  } else {
    *a = static_cast<unsigned>(__ldg(cu + s));
    *b = static_cast<unsigned>(__ldg(cu + s + 1));
  }
}

// Whether sequence bounds of seq_rows lie in rows [0, rows).
__device__ __forceinline__ bool bounds_ok(long long lo, long long hi, long long rows) {
  return hi >= lo && hi <= rows;
}

// Reports malformed offsets, whatever the call computes from them: thread i of n
// looks at every n-th sequence.
__device__ __forceinline__ void check_offsets(const int32_t* cu, int B, long long rows,
                                              long long i, long long n, unsigned* status) {
  for (long long s = i; s < B; s += n) {
    long long lo, hi;
    seq_rows(cu, (int)s, 0, &lo, &hi);
    if (!bounds_ok(lo, hi, rows) || (s == 0 && lo != 0) || (s == B - 1 && hi != rows))
      atomicOr(status, kDevBadSeqlens);
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
