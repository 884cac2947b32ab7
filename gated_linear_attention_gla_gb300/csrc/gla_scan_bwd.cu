// gla_scan_bwd.cu -- the gradients of the selective scan.
//
// With g_t = dy_t silu(z_t) (or dy_t), decay_t = exp(delta_t a) and e_t =
// dL/dh_t = c_t g_t + decay_{t+1} e_{t+1} (e behind the last token: the final
// state's gradient), per channel d and state n:
//     dc_t[n] = sum_d g_t h_t          db_t[n] = sum_d e_t delta_t u_t
//     w_t     = e_t decay_t h_{t-1}    da      = sum_t w_t delta_t
//     s1_t    = sum_n e_t b_t          s2_t    = sum_n a w_t
//     du_t    = delta_t s1_t + skip g_t
//     ddelta_t = s2_t + u_t s1_t,      ddt_t   = ddelta_t softplus'(dt_t + bias)
//     dskip = sum g u,  ddt_bias = sum ddt,  dz_t = dy_t y_t silu'(z_t),
//     d_init = decay_0 e_0
//
// Nothing of the forward pass is kept: the token axis is cut into chunks of 64
// and four launches run over (chunk, channel tile) blocks:
//   1. per chunk, the state it adds (h from zero), the gradient it passes to
//      the chunk before (e from zero, formed forwards with the running product
//      of the decays) and sum delta, whose exponential is the chunk's decay;
//   2. per (channel, n), both recurrences over the chunks: the state entering
//      and the gradient reaching every chunk;
//   3. per chunk: forwards once, keeping the state every 8 tokens, then
//      backwards in groups of 8 tokens whose states and decays are recomputed
//      into registers.  Sums over n are reduced over a channel's lanes, those
//      over d over the warp's channels, then over the warps in shared memory,
//      then written as one fp32 partial per channel tile;
//   4. the partials' sums (b, c over channel tiles; a, skip, dt_bias over chunks).
// No atomics: the same inputs give the same bits.  Bound: the CUDA cores and
// the exponential unit (three exponentials and ~17 multiply-adds per state and
// token), not HBM.
#include "gla_scan.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCH = 64;    // tokens per chunk
constexpr int kSub = 8;    // tokens per recomputed group
constexpr int kV = 4;      // adjacent channels per load

// Workspace, in floats: h and e [slots][D][NS], sums [slots][D] x 2, partials
// of db and dc [channel tiles][rows][2 NS].
struct Space {
  float *h, *e, *sum, *sum2, *part;
  size_t floats;
};
inline Space space_of(float* base, int B, long long rows, int D, int NS) {
  const size_t slots = (size_t)slots_of(B, rows, kCH);
  const size_t tiles = ((size_t)D * NS + 1023) / 1024;
  Space w;
  size_t at = 0;
  auto take = [&](size_t n) {
    float* q = base ? base + at : nullptr;
    at += (n + 63) / 64 * 64;
    return q;
  };
  w.h = take(slots * D * NS);
  w.e = take(slots * D * NS);
  w.sum = take(slots * D);
  w.sum2 = take(slots * D);
  w.part = take(tiles * (size_t)rows * 2 * NS);
  w.floats = at;
  return w;
}

template <typename IO>
__device__ __forceinline__ void load4(const void* base, long long row, long long stride, int ch,
                                      float (&x)[kV]) {
  unpack_as<IO, kV>(
      load_raw<IO, kV>((const IO*)base + row * stride + ch), x);
}

// delta, u and g of the chunk's pairs, and b, c, into shared memory (zeros for
// rows and channels that are not there); with kz, dy silu'(z) as well.
template <typename IO, int NS, int CT, bool KZ>
__device__ __forceinline__ void stage(const ScanBwdArgs& a, const Chunk& k, int d0,
                                      float (*s_delta)[CT], float (*s_u)[CT], float (*s_g)[CT],
                                      float (*s_k)[CT], float (*s_b)[NS], float (*s_c)[NS]) {
  const ScanArgs& p = a.f;
  constexpr int VPT = CT / kV, STEP = kThreads / VPT;
  const int vt = (int)threadIdx.x / VPT, vc = ((int)threadIdx.x % VPT) * kV;
  const bool von = d0 + vc < p.D;
  float bias[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) bias[i] = von && p.dt_bias ? __ldg(p.dt_bias + d0 + vc + i) : 0.f;
#pragma unroll
  for (int r = 0; r < kCH; r += STEP) {
    const int t = r + vt;
    if (t >= kCH) break;
    const long long row = k.t0 + t;
    float u[kV] = {}, dl[kV] = {}, g[kV] = {}, kz[kV] = {};
    if (row < k.t1 && von) {
      load4<IO>(p.u, row, p.u_stride, d0 + vc, u);
      load4<IO>(p.dt, row, p.dt_stride, d0 + vc, dl);
      load4<IO>(a.d_out, row, p.D, d0 + vc, g);
      float z[kV];
      if (p.z) load4<IO>(p.z, row, p.z_stride, d0 + vc, z);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        dl[i] += bias[i];
        if (p.softplus) dl[i] = softplus(dl[i]);
        if (p.z) {
          const float sg = sigmoid(z[i]);
          if (KZ) kz[i] = g[i] * sg * fmaf(z[i], 1.f - sg, 1.f);
          g[i] *= z[i] * sg;
        }
      }
    }
    *reinterpret_cast<float4*>(&s_delta[t][vc]) = make_float4(dl[0], dl[1], dl[2], dl[3]);
    *reinterpret_cast<float4*>(&s_u[t][vc]) = make_float4(u[0], u[1], u[2], u[3]);
    *reinterpret_cast<float4*>(&s_g[t][vc]) = make_float4(g[0], g[1], g[2], g[3]);
    if (KZ) *reinterpret_cast<float4*>(&s_k[t][vc]) = make_float4(kz[0], kz[1], kz[2], kz[3]);
  }
  for (int i = threadIdx.x; i < kCH * NS; i += kThreads) {
    const long long row = k.t0 + i / NS;
    float b = 0.f, c = 0.f;
    if (row < k.t1) {
      b = to_f32(((const IO*)p.b)[row * p.b_stride + i % NS]);
      c = to_f32(((const IO*)p.c)[row * p.c_stride + i % NS]);
    }
    s_b[i / NS][i % NS] = b;
    s_c[i / NS][i % NS] = c;
  }
}

template <int NS> __host__ __device__ constexpr int channel_tile() { return 1024 / NS; }

// 1. What each chunk adds to the state and to the gradient before it.
template <typename IO, int NS>
__global__ void __launch_bounds__(kThreads) chunk_sums_kernel(ScanBwdArgs a, Space w) {
  constexpr int LPC = NS / 4, CT = channel_tile<NS>();
  const ScanArgs& p = a.f;
  extern __shared__ __align__(16) unsigned char smem[];
  auto s_delta = reinterpret_cast<float (*)[CT]>(smem);
  auto s_u = s_delta + kCH;
  auto s_g = s_u + kCH;
  auto s_b = reinterpret_cast<float (*)[NS]>(s_g + kCH);
  auto s_c = s_b + kCH;
  const int tiles = (p.D + CT - 1) / CT;
  const long long slot = blockIdx.x / tiles;
  const int d0 = (int)(blockIdx.x % tiles) * CT;
  const Chunk k = chunk_of_slot(p, slot, kCH);
  if (!k.ok) return;
  const int q = threadIdx.x % LPC, lc = threadIdx.x / LPC, ch = d0 + lc;
  stage<IO, NS, CT, false>(a, k, d0, s_delta, s_u, s_g, nullptr, s_b, s_c);
  float a2[4] = {}, h[4] = {}, e[4] = {}, run[4] = {1.f, 1.f, 1.f, 1.f}, sum = 0.f;
  if (ch < p.D) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p.a + (long long)ch * NS) + q);
    a2[0] = x.x * kLog2e; a2[1] = x.y * kLog2e; a2[2] = x.z * kLog2e; a2[3] = x.w * kLog2e;
  }
  __syncthreads();
  const int len = (int)(k.t1 - k.t0);
#pragma unroll 4
  for (int t = 0; t < len; ++t) {
    const float dl = s_delta[t][lc], du = dl * s_u[t][lc], g = s_g[t][lc];
    const float4 b4 = *reinterpret_cast<const float4*>(&s_b[t][q * 4]);
    const float4 c4 = *reinterpret_cast<const float4*>(&s_c[t][q * 4]);
    const float b[4] = {b4.x, b4.y, b4.z, b4.w}, c[4] = {c4.x, c4.y, c4.z, c4.w};
    sum += dl;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float decay = ex2(dl * a2[j]);
      h[j] = fmaf(decay, h[j], du * b[j]);
      run[j] *= decay;
      e[j] = fmaf(run[j] * c[j], g, e[j]);
    }
  }
  if (ch < p.D) {
    const long long at = (slot * p.D + ch) * NS + q * 4;
    *reinterpret_cast<float4*>(w.h + at) = make_float4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<float4*>(w.e + at) = make_float4(e[0], e[1], e[2], e[3]);
    if (q == 0) w.sum[slot * p.D + ch] = sum;
  }
}

// 2. The state entering each chunk (blockIdx.y 0) and the gradient reaching its
// last token from behind (blockIdx.y 1), in place; d_init.
__global__ void __launch_bounds__(128)
chunk_scan_kernel(ScanBwdArgs a, Space w, long long slots) {
  const ScanArgs& p = a.f;
  const int quads = p.NS / 4;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long per = (long long)p.D * quads;
  if (i >= per * p.B) return;
  const int s = (int)(i / per);
  const long long in = i % per;  // channel * quads + quad
  const int ch = (int)(in / quads);
  long long lo, hi;
  if (!seq_ok(p, s, in == 0, &lo, &hi)) return;
  const long long f = first_slot(p, s, kCH);
  const long long n = min((hi - lo + kCH - 1) / kCH, slots - f);
  float4 x = __ldg(reinterpret_cast<const float4*>(p.a) + in);
  x.x *= kLog2e; x.y *= kLog2e; x.z *= kLog2e; x.w *= kLog2e;
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool back = blockIdx.y != 0;
  const float* start = back ? a.d_final_state : p.init_state;
  if (start) run = reinterpret_cast<const float4*>(start)[(long long)s * per + in];
  scan_chunks(reinterpret_cast<float4*>(back ? w.e : w.h), w.sum, x, f, n, per, in, p.D, ch, back,
              &run);
  if (back && a.d_init_state) reinterpret_cast<float4*>(a.d_init_state)[(long long)s * per + in] = run;
}

// The sums of v[0 .. 8) over the lanes that differ in the bits LPC .. 16,
// scattered: afterwards a lane holds N of them, v[0 .. N), from index *first.
template <int OFF, int LPC, int N>
__device__ __forceinline__ void reduce_channels(float (&v)[8], int lane, int* first) {
  if constexpr (OFF >= LPC) {
    if constexpr (N > 1) {
      const bool up = (lane & OFF) != 0;
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        const float give = up ? v[k] : v[k + N / 2];
        const float keep = up ? v[k + N / 2] : v[k];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, give, OFF);
      }
      if (up) *first += N / 2;
      reduce_channels<OFF / 2, LPC, N / 2>(v, lane, first);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], OFF);
      reduce_channels<OFF / 2, LPC, 1>(v, lane, first);
    }
  }
}

// 3. The chunk's gradients.
template <typename IO, typename OUT, int NS>
__global__ void __launch_bounds__(kThreads, 2) chunk_grads_kernel(ScanBwdArgs a, Space w) {
  constexpr int LPC = NS / 4, CT = channel_tile<NS>(), G = 32 / LPC;
  constexpr int HELD = G >= 8 ? 1 : 8 / G;    // sums over d that a lane ends up with
  constexpr int kShare = LPC > 4 ? LPC / 4 : 1;  // lanes that share a sum over n
  const ScanArgs& p = a.f;
  extern __shared__ __align__(16) unsigned char smem[];
  auto s_delta = reinterpret_cast<float (*)[CT]>(smem);  // later ddt
  auto s_u = s_delta + kCH;                               // later du
  auto s_g = s_u + kCH;
  auto s_k = s_g + kCH;                                   // later dz
  auto s_b = reinterpret_cast<float (*)[NS]>(s_k + kCH);
  auto s_c = s_b + kCH;
  auto s_h = reinterpret_cast<float4*>(s_c + kCH);        // [kCH / kSub][kThreads]
  auto s_red = reinterpret_cast<float (*)[kSub][2 * NS]>(s_h + kCH / kSub * kThreads);  // [kWarps]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = (p.D + CT - 1) / CT, tile = (int)(blockIdx.x % tiles);
  const long long slot = blockIdx.x / tiles;
  const long long rows = p.cu_seqlens ? (long long)p.T : (long long)p.B * p.T;
  const int d0 = tile * CT;
  const int q = tid % LPC, lc = tid / LPC, ch = d0 + lc;
  const bool on = ch < p.D;
  const long long at = (slot * p.D + ch) * NS + q * 4;
  const Chunk k = chunk_of_slot(p, slot, kCH);
  if (!k.ok) {  // no chunk: its partials count as zero
    if (on) {
      *reinterpret_cast<float4*>(w.h + at) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q == 0) w.sum[slot * p.D + ch] = w.sum2[slot * p.D + ch] = 0.f;
    }
    return;
  }
  stage<IO, NS, CT, true>(a, k, d0, s_delta, s_u, s_g, s_k, s_b, s_c);
  float a2[4] = {}, h[4] = {}, e[4] = {}, da[4] = {};
  float skip = 0.f, dskip = 0.f, dbias = 0.f;
  if (on) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p.a + (long long)ch * NS) + q);
    a2[0] = x.x * kLog2e; a2[1] = x.y * kLog2e; a2[2] = x.z * kLog2e; a2[3] = x.w * kLog2e;
    const float4 y = *reinterpret_cast<const float4*>(w.h + at);
    h[0] = y.x; h[1] = y.y; h[2] = y.z; h[3] = y.w;
    const float4 v = *reinterpret_cast<const float4*>(w.e + at);
    e[0] = v.x; e[1] = v.y; e[2] = v.z; e[3] = v.w;
    if (p.skip) skip = __ldg(p.skip + ch);
  }
  __syncthreads();
  const int len = (int)(k.t1 - k.t0);
  const int groups = (len + kSub - 1) / kSub;

  // forwards, keeping the state in front of every group (rows behind the
  // sequence have delta = 0: decay 1, no drive)
  for (int gr = 0; gr < groups; ++gr) {
    s_h[gr * kThreads + tid] = make_float4(h[0], h[1], h[2], h[3]);
    if (gr + 1 == groups) break;
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      const int t = gr * kSub + i;
      const float dl = s_delta[t][lc], du = dl * s_u[t][lc];
      const float4 b4 = *reinterpret_cast<const float4*>(&s_b[t][q * 4]);
      const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = fmaf(ex2(dl * a2[j]), h[j], du * b[j]);
    }
  }
  // backwards
  for (int gr = groups - 1; gr >= 0; --gr) {
    float hs[kSub + 1][4], ds[kSub][4];
    {
      const float4 x = s_h[gr * kThreads + tid];
      hs[0][0] = x.x; hs[0][1] = x.y; hs[0][2] = x.z; hs[0][3] = x.w;
    }
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      const int t = gr * kSub + i;
      const float dl = s_delta[t][lc], du = dl * s_u[t][lc];
      const float4 b4 = *reinterpret_cast<const float4*>(&s_b[t][q * 4]);
      const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ds[i][j] = ex2(dl * a2[j]);
        hs[i + 1][j] = fmaf(ds[i][j], hs[i][j], du * b[j]);
      }
    }
#pragma unroll
    for (int half = kSub / 4 - 1; half >= 0; --half) {
      float s1[4], s2[4], y[4];
      float vb[8], vc[8];
#pragma unroll
      for (int x = 3; x >= 0; --x) {
        const int i = half * 4 + x, t = gr * kSub + i;
        const float dl = s_delta[t][lc], du = dl * s_u[t][lc], g = s_g[t][lc];
        const float4 b4 = *reinterpret_cast<const float4*>(&s_b[t][q * 4]);
        const float4 c4 = *reinterpret_cast<const float4*>(&s_c[t][q * 4]);
        const float b[4] = {b4.x, b4.y, b4.z, b4.w}, c[4] = {c4.x, c4.y, c4.z, c4.w};
        s1[x] = s2[x] = y[x] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[j] = fmaf(c[j], g, e[j]);
          vc[(x & 1) * 4 + j] = g * hs[i + 1][j];
          vb[(x & 1) * 4 + j] = du * e[j];
          s1[x] = fmaf(e[j], b[j], s1[x]);
          y[x] = fmaf(c[j], hs[i + 1][j], y[x]);
          e[j] *= ds[i][j];
          const float wj = e[j] * hs[i][j];
          da[j] = fmaf(dl, wj, da[j]);
          s2[x] = fmaf(a2[j], wj, s2[x]);
        }
        if ((x & 1) == 0) {  // tokens i and i + 1
          int fb = 0, fc = 0;
          reduce_channels<16, LPC, 8>(vb, lane, &fb);
          reduce_channels<16, LPC, 8>(vc, lane, &fc);
          if (G <= 8 || (lane & LPC) == 0) {
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
              s_red[warp][i + (fb + m) / 4][q * 4 + (fb + m) % 4] = vb[m];
              s_red[warp][i + (fc + m) / 4][NS + q * 4 + (fc + m) % 4] = vc[m];
            }
          }
        }
      }
      int first;
      reduce4<LPC>(s1, q, &first);
      reduce4<LPC>(s2, q, &first);
      reduce4<LPC>(y, q, &first);
      __syncwarp();  // the channel's lanes have read delta, u and g
#pragma unroll
      for (int m = 0; m < (LPC == 2 ? 2 : 1); ++m) {
        const int t = gr * kSub + half * 4 + first + m;
        if (t < len && q % kShare == 0) {
          const float dl = s_delta[t][lc], u = s_u[t][lc], g = s_g[t][lc];
          float ddt = fmaf(kLn2, s2[m], u * s1[m]);
          // softplus'(x) = 1 - e^-softplus(x)
          if (p.softplus) ddt *= -expm1f(-dl);
          dskip = fmaf(g, u, dskip);
          dbias += ddt;
          s_delta[t][lc] = ddt;
          s_u[t][lc] = fmaf(dl, s1[m], skip * g);
          s_k[t][lc] *= fmaf(skip, u, y[m]);
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < kSub * 2 * NS; i += kThreads) {
      const int t = i / (2 * NS), col = i % (2 * NS);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) sum += s_red[v][t][col];
      const long long row = k.t0 + gr * kSub + t;
      if (row < k.t1) w.part[((long long)tile * rows + row) * 2 * NS + col] = sum;
    }
    __syncthreads();
  }
  // this chunk's share of da, dskip, ddt_bias over the inputs it has consumed
#pragma unroll
  for (int off = LPC / 2; off > 0; off >>= 1) {
    dskip += __shfl_xor_sync(0xffffffffu, dskip, off);
    dbias += __shfl_xor_sync(0xffffffffu, dbias, off);
  }
  if (on) {
    *reinterpret_cast<float4*>(w.h + at) = make_float4(da[0], da[1], da[2], da[3]);
    if (q == 0) {
      w.sum[slot * p.D + ch] = dskip;
      w.sum2[slot * p.D + ch] = dbias;
    }
  }
  // du, ddt, dz in rows of adjacent channels (the last group's barrier precedes)
  constexpr int VPT = CT / kV, STEP = kThreads / VPT;
  const int vt = tid / VPT, vc = (tid % VPT) * kV;
  if (d0 + vc < p.D) {
    for (int t = vt; t < len; t += STEP) {
      const long long o = (k.t0 + t) * p.D + d0 + vc;
      auto put = [&](void* to, const float* from) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        const float y[kV] = {x.x, x.y, x.z, x.w};
        store_raw<OUT, kV>((OUT*)to + o, pack_as<OUT, kV>(y));
      };
      put(a.du, &s_u[t][vc]);
      put(a.ddt, &s_delta[t][vc]);
      if (a.dz) put(a.dz, &s_k[t][vc]);
    }
  }
}

// 4a. db and dc: the channel tiles' partials.
template <typename OUT>
__global__ void __launch_bounds__(256)
sum_tiles_kernel(ScanBwdArgs a, Space w, int tiles, long long rows) {
  const int NS = a.f.NS;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long n = rows * 2 * NS;
  if (i >= n) return;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  int t = 0;
  for (; t + 4 <= tiles; t += 4)
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += w.part[(t + u) * n + i];
  for (; t < tiles; ++t) s[0] += w.part[t * n + i];
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  const long long row = i / (2 * NS);
  const int col = (int)(i % (2 * NS));
  if (col < NS) ((OUT*)a.db)[row * NS + col] = from_f32<OUT>(sum);
  else ((OUT*)a.dc)[row * NS + col - NS] = from_f32<OUT>(sum);
}

// 4b. da, dskip and ddt_bias: the chunks' partials.
__global__ void __launch_bounds__(256)
sum_chunks_kernel(ScanBwdArgs a, Space w, long long slots) {
  const long long D = a.f.D, DN = D * a.f.NS;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const float* from;
  float* to;
  long long step;
  if (i < DN) { from = w.h + i; to = a.da + i; step = DN; }
  else if (i < DN + D) { from = w.sum + i - DN; to = a.dskip ? a.dskip + i - DN : nullptr; step = D; }
  else if (i < DN + 2 * D) {
    from = w.sum2 + i - DN - D;
    to = a.ddt_bias ? a.ddt_bias + i - DN - D : nullptr;
    step = D;
  } else return;
  if (!to) return;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  long long t = 0;
  for (; t + 4 <= slots; t += 4)
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += from[(t + u) * step];
  for (; t < slots; ++t) s[0] += from[t * step];
  *to = (s[0] + s[1]) + (s[2] + s[3]);
}

template <typename K> cudaError_t opt_in(K kernel, int bytes) {
  return bytes > 48 * 1024
             ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
             : cudaSuccess;
}

template <typename IO, typename OUT, int NS>
cudaError_t launch_typed(const ScanBwdArgs& a, void* workspace, cudaStream_t stream) {
  constexpr int CT = channel_tile<NS>();
  const ScanArgs& p = a.f;
  const long long rows = p.cu_seqlens ? (long long)p.T : (long long)p.B * p.T;
  const long long slots = slots_of(p.B, rows, kCH);
  const int tiles = (p.D + CT - 1) / CT;
  const Space w = space_of(static_cast<float*>(workspace), p.B, rows, p.D, NS);
  constexpr int staged = 2 * kCH * NS * 4;
  constexpr int smem1 = 3 * kCH * CT * 4 + staged;
  constexpr int smem3 = 4 * kCH * CT * 4 + staged + kCH / kSub * kThreads * 16 +
                        kWarps * kSub * 2 * NS * 4;
  static_assert(smem3 <= 227 * 1024, "shared memory of a block");
  cudaError_t e = opt_in(chunk_sums_kernel<IO, NS>, smem1);
  if (e == cudaSuccess) e = opt_in(chunk_grads_kernel<IO, OUT, NS>, smem3);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(slots * tiles);
  if (rows > 0) chunk_sums_kernel<IO, NS><<<grid, kThreads, smem1, stream>>>(a, w);
  const long long per = (long long)p.B * p.D * (NS / 4);
  if (p.B > 0) {
    chunk_scan_kernel<<<dim3((unsigned)((per + 127) / 128), 2), 128, 0, stream>>>(a, w, slots);
    chunk_grads_kernel<IO, OUT, NS><<<grid, kThreads, smem3, stream>>>(a, w);
  }
  if (rows > 0)
    sum_tiles_kernel<OUT><<<(unsigned)((rows * 2 * NS + 255) / 256), 256, 0, stream>>>(a, w, tiles,
                                                                                      rows);
  const long long n = (long long)p.D * (NS + 2);
  sum_chunks_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(a, w, slots);
  return cudaGetLastError();
}

template <typename IO, typename OUT>
cudaError_t launch_io(const ScanBwdArgs& a, void* workspace, cudaStream_t stream) {
  switch (a.f.NS) {
    case 8: return launch_typed<IO, OUT, 8>(a, workspace, stream);
    case 16: return launch_typed<IO, OUT, 16>(a, workspace, stream);
    case 32: return launch_typed<IO, OUT, 32>(a, workspace, stream);
    default: return launch_typed<IO, OUT, 64>(a, workspace, stream);
  }
}

}  // namespace

size_t scan_bwd_workspace(int B, long long rows, int D, int NS) {
  return space_of(nullptr, B, rows, D, NS).floats * 4;
}

cudaError_t launch_scan_bwd(const ScanBwdArgs& a, void* workspace, cudaStream_t stream) {
  if (a.f.fp32_io) return launch_io<float, float>(a, workspace, stream);
  if (a.f.fp32_out) return launch_io<__nv_bfloat16, float>(a, workspace, stream);
  return launch_io<__nv_bfloat16, __nv_bfloat16>(a, workspace, stream);
}

}  // namespace gla
