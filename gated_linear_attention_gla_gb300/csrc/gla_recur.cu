// gla_recur.cu -- the gated linear recurrence: how a call is split, and single tokens.
#include "gla_recur.cuh"

namespace gla {
namespace recur {

Split split(int B, int T, int D, bool packed, int run, int most, int blocks) {
  Split p;
  p.cols = (D + kChans - 1) / kChans;
  // Short sequences share a group, so that a step's runs are filled, but no fewer groups than one
  // wave of blocks (2048 channels: 170 sequences of 48 tokens 90 us, 122 us alone; 16 of 32 tokens by
  // fours 9.7 us, all together 13.0 us; 64 of 128 tokens alone 66 us, 85 us by fours, their gradients
  // 177 and 168 us)
  p.spg = 1;
  if (T > 0 && T < 128) {
    const int groups = p.cols < 152 ? 152 / p.cols : 1;  // of one wave of blocks
    const int share = B / groups + (B % groups != 0);
    p.spg = (512 + T - 1) / T;
    if (p.spg > share) p.spg = share;
  }
  if (packed) p.spg = 0;
  if (p.spg > B) p.spg = B;
  p.groups = packed ? 1 : ((long long)B + p.spg - 1) / (p.spg > 0 ? p.spg : 1);
  p.rows = packed ? T : (long long)p.spg * T;
  const long long units = (long long)p.cols * p.groups;
  // as many blocks as the SMs hold, while every block has tokens (2048 channels, 4 sequences of 256
  // tokens 8.9 us, with twice the blocks 15.4 us)
  p.warps = most;
  p.cluster = 1;
  while (p.cluster < kMaxCluster && units * p.cluster * 2 <= blocks * 152 &&
         (long long)p.cluster * p.warps * run < p.rows)
    p.cluster *= 2;
  while (p.warps > 1 && (long long)(p.warps / 2) * p.cluster * run >= p.rows) p.warps /= 2;
  return p;
}

namespace {

template <typename T, typename OT>
__global__ void __launch_bounds__(256) recur_step_kernel(RecurStepArgs a) {
  after_previous();
  start_next();
  const long long n = (long long)blockIdx.z * gridDim.y + blockIdx.y;
  const int c = ((int)blockIdx.x * (int)blockDim.x + (int)threadIdx.x) * 4;
  if (c >= a.D || n >= a.N) return;
  long long from = n, to = n;
  if (a.slots != nullptr) {
    const int f = __ldg(a.slots + n), t = a.out_slots ? __ldg(a.out_slots + n) : f;
    if (f < 0 || t < 0) return;  // a padding row
    if (f >= a.num_slots || t >= a.num_slots) {
      if (threadIdx.x == 0) atomicOr(a.status, kDevBadSeqlens);
      return;
    }
    from = f;
    to = t;
  }
  constexpr bool EXACT = sizeof(T) == 4;
  f32x2 x[2], f[2], i[2] = {}, z[2] = {};
  unpack_pairs<T, 4>(load_raw<T, 4>((const T*)a.x + n * a.x_stride + c), x);
  unpack_pairs<T, 4>(load_raw<T, 4>((const T*)a.f + n * a.f_stride + c), f);
  if (a.i) unpack_pairs<T, 4>(load_raw<T, 4>((const T*)a.i + n * a.i_stride + c), i);
  if (a.z) unpack_pairs<T, 4>(load_raw<T, 4>((const T*)a.z + n * a.z_stride + c), z);
  float4 dec = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.decay) dec = __ldg(reinterpret_cast<const float4*>(a.decay + c));
  const float4 old = *reinterpret_cast<const float4*>(a.state + from * a.D + c);
  const f32x2 h0[2] = {make_float2(old.x, old.y), make_float2(old.z, old.w)};
  const f32x2 d[2] = {decay_log2(make_float2(dec.x, dec.y)), decay_log2(make_float2(dec.z, dec.w))};
  f32x2 h[2];
  float y[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Gate g = a.decay ? gates<EXACT, true, true, false, false>(f[k], i[k], d[k], a.unit)
                           : gates<EXACT, false, true, false, false>(f[k], i[k], d[k], a.unit);
    h[k] = fma2(g.a, h0[k], mul2(a.i ? mul2(g.m, g.si) : g.m, x[k]));
    f32x2 v = h[k];
    if (a.z) {
      f32x2 sz;
      sigmoids<EXACT>(z[k], &sz, nullptr);
      v = mul2(v, mul2(z[k], sz));
    }
    y[2 * k] = v.x;
    y[2 * k + 1] = v.y;
  }
  *reinterpret_cast<float4*>(a.state + to * a.D + c) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
  store_raw<OT, 4>((OT*)a.out + n * a.D + c, pack_as<OT, 4>(y));
}

}  // namespace
}  // namespace recur

cudaError_t launch_recur_fwd(const RecurArgs& a, cudaStream_t stream) {
  return a.fp32_io ? recur::fwd_f32(a, stream) : recur::fwd_bf16(a, stream);
}

cudaError_t launch_recur_step(const RecurStepArgs& a, cudaStream_t stream) {
  const int vecs = a.D / 4;
  const int threads = vecs >= 128 ? 128 : (vecs + 31) / 32 * 32;
  const unsigned ny = a.N < 65535 ? (unsigned)a.N : 65535u;  // (2^31 - 1 rows are 32769 times as many)
  const dim3 grid((unsigned)((vecs + threads - 1) / threads), ny, (unsigned)((a.N + ny - 1) / ny));
  using bf16 = __nv_bfloat16;
  return launch_after(a.fp32_io    ? recur::recur_step_kernel<float, float>
                      : a.fp32_out ? recur::recur_step_kernel<bf16, float>
                                   : recur::recur_step_kernel<bf16, bf16>,
                      grid, dim3(threads), 0, stream, a);
}

}  // namespace gla
