// gla_scan_step.cu -- one token of the selective scan for N sequences.
//
//     delta = softplus(dt + dt_bias)
//     h'[d][n] = exp(delta a[d][n]) h[d][n] + delta u b[n]        (fp32 page)
//     y[d] = (sum_n c[n] h'[d][n] + skip[d] u) * silu(z)
//
// The step streams the state: 8 bytes per (channel, n) against four inputs and
// one output per channel, so HBM bounds it.  NS / 4 adjacent lanes own a
// channel, four states (16 bytes) each; a block owns 1024 / NS channels and
// walks kSeqs sequences, whose pages are all loaded before the first is used;
// a, skip and dt_bias are read once per block.
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;

template <typename IO, typename OUT, int NS, int SEQS>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanStepArgs p) {
  constexpr int LPC = NS / 4;
  const int q = threadIdx.x % LPC;
  const int d = (int)blockIdx.x * (kThreads / LPC) + (int)threadIdx.x / LPC;
  const bool on = d < p.D;
  const int ch = on ? d : 0;  // lanes past the end still join the sums
  const long long n0 = ((long long)blockIdx.y + (long long)blockIdx.z * gridDim.y) * SEQS;

  long long from[SEQS], to[SEQS];
  float4 h[SEQS];
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    const long long n = n0 + i;
    from[i] = to[i] = n < p.N ? n : -1;
    if (p.slots != nullptr && n < p.N) {
      const int f = __ldg(p.slots + n), t = p.out_slots ? __ldg(p.out_slots + n) : f;
      const bool bad = f >= p.num_slots || t >= p.num_slots;
      if (bad && f >= 0 && t >= 0 && threadIdx.x == 0) atomicOr(p.status, kDevBadSeqlens);
      from[i] = bad || f < 0 || t < 0 ? -1 : f;
      to[i] = t;
    }
    h[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (from[i] >= 0 && on)
      h[i] = __ldcs(reinterpret_cast<const float4*>(p.state + (from[i] * p.D + ch) * NS) + q);
  }
  const float4 a = __ldg(reinterpret_cast<const float4*>(p.a + (long long)ch * NS) + q);
  const float bias = p.dt_bias ? __ldg(p.dt_bias + ch) : 0.f;
  const float skip = p.skip ? __ldg(p.skip + ch) : 0.f;

#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    if (from[i] < 0) continue;  // uniform over the block
    const long long n = n0 + i;
    const float u = to_f32(((const IO*)p.u)[n * p.u_stride + ch]);
    float delta = to_f32(((const IO*)p.dt)[n * p.dt_stride + ch]) + bias;
    if (p.softplus) delta = softplus(delta);
    float b[4], c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      b[k] = to_f32(((const IO*)p.b)[n * p.b_stride + q * 4 + k]);
      c[k] = to_f32(((const IO*)p.c)[n * p.c_stride + q * 4 + k]);
    }
    const float w = delta * u, e = delta * kLog2e;
    float4 x = h[i];
    x.x = fmaf(ex2(e * a.x), x.x, w * b[0]);
    x.y = fmaf(ex2(e * a.y), x.y, w * b[1]);
    x.z = fmaf(ex2(e * a.z), x.z, w * b[2]);
    x.w = fmaf(ex2(e * a.w), x.w, w * b[3]);
    if (on) __stcs(reinterpret_cast<float4*>(p.state + (to[i] * p.D + ch) * NS) + q, x);
    float y = fmaf(c[0], x.x, fmaf(c[1], x.y, fmaf(c[2], x.z, c[3] * x.w)));
#pragma unroll
    for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    if (on && q == 0) {
      y = fmaf(skip, u, y);
      if (p.z) y *= silu(to_f32(((const IO*)p.z)[n * p.z_stride + ch]));
      ((OUT*)p.out)[n * p.D + ch] = from_f32<OUT>(y);
    }
  }
}

template <typename IO, typename OUT, int NS, int SEQS>
cudaError_t launch_seqs(const ScanStepArgs& a, cudaStream_t stream) {
  constexpr int kChannels = kThreads / (NS / 4);
  const long long groups = ((long long)a.N + SEQS - 1) / SEQS;
  const unsigned ny = groups < 32768 ? (unsigned)groups : 32768u;
  const dim3 grid((unsigned)((a.D + kChannels - 1) / kChannels), ny,
                  (unsigned)((groups + ny - 1) / ny));
  scan_step_kernel<IO, OUT, NS, SEQS><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename IO, typename OUT>
cudaError_t launch_io(const ScanStepArgs& a, cudaStream_t stream) {
  switch (a.NS) {
    case 8: return launch_seqs<IO, OUT, 8, 4>(a, stream);
    case 16: return launch_seqs<IO, OUT, 16, 4>(a, stream);
    case 32: return launch_seqs<IO, OUT, 32, 4>(a, stream);
    default: return launch_seqs<IO, OUT, 64, 4>(a, stream);
  }
}

}  // namespace

cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t stream) {
  if (a.fp32_io) return launch_io<float, float>(a, stream);
  if (a.fp32_out) return launch_io<__nv_bfloat16, float>(a, stream);
  return launch_io<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

}  // namespace gla
