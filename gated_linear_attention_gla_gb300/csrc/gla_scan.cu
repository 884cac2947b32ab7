// gla_scan.cu -- the selective scan over prompts (dense or packed).
//
//     delta = softplus(dt + dt_bias)
//     h_t[d][n] = exp(delta_t[d] a[d][n]) h_{t-1}[d][n] + delta_t[d] u_t[d] b_t[n]
//     y_t[d] = (sum_n c_t[n] h_t[d][n] + skip[d] u_t[d]) * silu(z_t[d])
//
// Every (channel, n) has a decay of its own at every token, so no product of
// matrices forms the in-chunk part (as it does in chunk_fwd): the work is NS
// exponentials and 4 NS multiply-adds per token and channel, on the CUDA cores.
//
// NS / 4 adjacent lanes own a channel, four states each in registers; a block
// of 8 warps owns a tile of 1024 / NS channels of one sequence and walks its tokens
// in tiles of 1024 (token, channel) pairs.  Per tile every thread turns four
// pairs into (delta, delta u) in shared memory, loaded a tile ahead; the
// lanes then run the recurrence, the sum over n is reduced over the lanes of
// a channel for four tokens at once, and the thread that holds u and z of a
// pair finishes and stores it.  One barrier per tile (double-buffered).
#include "gla_scan.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;
constexpr int kPairs = 1024;  // (token, channel) pairs of a tile
constexpr int kV = 4;         // pairs per thread: adjacent channels of a token

template <typename IO, typename OUT, int NS>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(ScanArgs p) {
  constexpr int LPC = NS / 4;             // lanes per channel
  constexpr int CT = kThreads / LPC;      // channels per block
  constexpr int TT = kPairs / CT;         // tokens per tile
  constexpr int VPT = CT / kV;            // threads per token of a tile
  constexpr int BC = (TT * NS + kThreads - 1) / kThreads;  // b (and c) elements per thread

  extern __shared__ __align__(16) unsigned char smem[];
  auto s_d = reinterpret_cast<float2 (*)[TT][CT]>(smem);  // [2]: delta, delta u
  auto s_b = reinterpret_cast<float (*)[TT][NS]>(smem + 2 * kPairs * 8);
  auto s_c = s_b + 2;
  auto s_y = reinterpret_cast<float (*)[TT][CT]>(s_c + 2);

  const int tid = threadIdx.x;
  const int q = tid % LPC, lc = tid / LPC;        // the recurrence's role
  const int tiles = (p.D + CT - 1) / CT;
  const int d0 = (int)(blockIdx.x % tiles) * CT;
  const int ch = min(d0 + lc, p.D - 1);
  const int vt = tid / VPT, vc = (tid % VPT) * kV;  // the pairs' role
  const bool von = d0 + vc < p.D;
  const int s = (int)(blockIdx.x / tiles);
  const long long rows = p.cu_seqlens ? (long long)p.T : (long long)p.B * p.T;

  long long lo, hi;
  seq_rows(p.cu_seqlens, s, p.T, &lo, &hi);
  if (lo < 0 || hi < lo || hi > rows || (p.cu_seqlens && (__ldg(p.cu_seqlens) != 0 ||
                                                         __ldg(p.cu_seqlens + p.B) != rows))) {
    if (tid == 0) atomicOr(p.status, kDevBadSeqlens);
    return;
  }

  float a2[4], h[4];
  {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.a + (long long)ch * NS) + q);
    a2[0] = a.x * kLog2e; a2[1] = a.y * kLog2e; a2[2] = a.z * kLog2e; a2[3] = a.w * kLog2e;
    float4 h0 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.init_state)
      h0 = *(reinterpret_cast<const float4*>(p.init_state + ((long long)s * p.D + ch) * NS) + q);
    h[0] = h0.x; h[1] = h0.y; h[2] = h0.z; h[3] = h0.w;
  }
  float bias[kV], skip[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    bias[i] = von && p.dt_bias ? __ldg(p.dt_bias + d0 + vc + i) : 0.f;
    skip[i] = von && p.skip ? __ldg(p.skip + d0 + vc + i) : 0.f;
  }

  using R = Raw<IO, kV>;
  R ru = zero_raw<IO, kV>(), rdt = ru, rz = ru, fu = ru, fz = ru;  // next tile; tile to finish
  IO rb[BC], rc[BC];
  auto load = [&](long long t0) {
    const long long t = t0 + vt;
    ru = rdt = rz = zero_raw<IO, kV>();
    if (t < hi && von) {
      ru = *reinterpret_cast<const R*>((const IO*)p.u + t * p.u_stride + d0 + vc);
      rdt = *reinterpret_cast<const R*>((const IO*)p.dt + t * p.dt_stride + d0 + vc);
      if (p.z) rz = *reinterpret_cast<const R*>((const IO*)p.z + t * p.z_stride + d0 + vc);
    }
#pragma unroll
    for (int k = 0; k < BC; ++k) {
      const int i = tid + k * kThreads;
      const long long tb = t0 + i / NS;
      rb[k] = rc[k] = from_f32<IO>(0.f);
      if (i < TT * NS && tb < hi) {
        rb[k] = ((const IO*)p.b)[tb * p.b_stride + i % NS];
        rc[k] = ((const IO*)p.c)[tb * p.c_stride + i % NS];
      }
    }
  };
  auto finish = [&](long long t0, int buf) {  // y of the pairs whose u and z are in fu, fz
    const long long t = t0 + vt;
    if (t >= hi || !von) return;
    float u[kV], z[kV], y[kV];
    unpack_as<IO, kV>(fu, u);
    unpack_as<IO, kV>(fz, z);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      y[i] = fmaf(skip[i], u[i], s_y[buf][vt][vc + i]);
      if (p.z) y[i] *= silu(z[i]);
    }
    *reinterpret_cast<Raw<OUT, kV>*>((OUT*)p.out + t * p.D + d0 + vc) = pack_as<OUT, kV>(y);
  };

  load(lo);
  int buf = 0;
  for (long long t0 = lo; t0 < hi; t0 += TT, buf ^= 1) {
    {
      float u[kV], x[kV];
      unpack_as<IO, kV>(ru, u);
      unpack_as<IO, kV>(rdt, x);
      const bool in = t0 + vt < hi;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        float delta = x[i] + bias[i];
        if (p.softplus) delta = softplus(delta);
        // tokens behind the sequence: decay 1, no drive
        s_d[buf][vt][vc + i] = in ? make_float2(delta, delta * u[i]) : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < BC; ++k) {
        const int i = tid + k * kThreads;
        if (i < TT * NS) {
          (&s_b[buf][0][0])[i] = to_f32(rb[k]);
          (&s_c[buf][0][0])[i] = to_f32(rc[k]);
        }
      }
    }
    __syncthreads();
    if (t0 > lo) finish(t0 - TT, buf ^ 1);
    fu = ru;
    fz = rz;
    if (t0 + TT < hi) load(t0 + TT);
#pragma unroll 2
    for (int t4 = 0; t4 < TT; t4 += 4) {
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 dd = s_d[buf][t4 + k][lc];
        const float4 b = *reinterpret_cast<const float4*>(&s_b[buf][t4 + k][q * 4]);
        const float4 c = *reinterpret_cast<const float4*>(&s_c[buf][t4 + k][q * 4]);
        h[0] = fmaf(ex2(dd.x * a2[0]), h[0], dd.y * b.x);
        h[1] = fmaf(ex2(dd.x * a2[1]), h[1], dd.y * b.y);
        h[2] = fmaf(ex2(dd.x * a2[2]), h[2], dd.y * b.z);
        h[3] = fmaf(ex2(dd.x * a2[3]), h[3], dd.y * b.w);
        y[k] = fmaf(c.x, h[0], fmaf(c.y, h[1], fmaf(c.z, h[2], c.w * h[3])));
      }
      int first;
      reduce4<LPC>(y, q, &first);
      if constexpr (LPC == 2) {
        s_y[buf][t4 + first][lc] = y[0];
        s_y[buf][t4 + first + 1][lc] = y[1];
      } else {
        if (q % (LPC / 4) == 0) s_y[buf][t4 + first][lc] = y[0];
      }
    }
  }
  __syncthreads();
  if (hi > lo) finish(lo + (hi - lo - 1) / TT * TT, buf ^ 1);
  if (p.final_state && d0 + lc < p.D)
    *(reinterpret_cast<float4*>(p.final_state + ((long long)s * p.D + d0 + lc) * NS) + q) =
        make_float4(h[0], h[1], h[2], h[3]);
}

template <typename IO, typename OUT, int NS>
cudaError_t launch_typed(const ScanArgs& a, cudaStream_t stream) {
  constexpr int CT = kThreads / (NS / 4), TT = kPairs / CT;
  constexpr int smem = 2 * (kPairs * 12 + 2 * TT * NS * 4);
  auto kernel = scan_fwd_kernel<IO, OUT, NS>;
  if constexpr (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)((long long)((a.D + CT - 1) / CT) * a.B), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename IO, typename OUT>
cudaError_t launch_io(const ScanArgs& a, cudaStream_t stream) {
  switch (a.NS) {
    case 8: return launch_typed<IO, OUT, 8>(a, stream);
    case 16: return launch_typed<IO, OUT, 16>(a, stream);
    case 32: return launch_typed<IO, OUT, 32>(a, stream);
    default: return launch_typed<IO, OUT, 64>(a, stream);
  }
}

}  // namespace

size_t scan_fwd_workspace(int, long long, int, int) { return 0; }

cudaError_t launch_scan_fwd(const ScanArgs& a, void*, cudaStream_t stream) {
  if (a.fp32_io) return launch_io<float, float>(a, stream);
  if (a.fp32_out) return launch_io<__nv_bfloat16, float>(a, stream);
  return launch_io<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

}  // namespace gla
