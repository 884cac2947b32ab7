// gla_conv_bwd.cu -- the gradients of the short causal convolution.
//
// With p recomputed and dp_t = dy_t silu'(p_t) (or dy_t):
//     dx_t[d]        = sum_j weight[d][W - 1 - j] dp_{t+j}[d]      (t + j inside the sequence)
//     d_weight[d][k] = sum_t dp_t[d] x_{t-(W-1)+k}[d],   d_bias[d] = sum_t dp_t[d]
// The final state is a copy of the last W - 1 rows, so its gradient adds to
// theirs; the initial state's rows are rows in front of the sequence.
//
// One pass over x and dy: a thread owns 4 adjacent channels and a run of 32
// rows, with the last W - 1 rows of x and of dp in registers; dx of a row
// leaves W - 1 rows later, so a run reads W - 1 rows past its end (their dp
// only).  The weight's gradient is summed in registers over the run, in shared
// memory over a block's 8 runs, and written as one fp32 partial per block; a
// second launch sums the partials in block order.  No atomics: the same inputs
// give the same bits.
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kV = 4;         // channels per thread
constexpr int kRun = 32;      // rows per thread
constexpr int kGroups = 8;    // runs per block
constexpr int kUnroll = 4;    // rows in flight

template <bool SILU> __device__ __forceinline__ float d_act(float p) {
  if (!SILU) return 1.f;
  const float s = sigmoid(p);
  return s * fmaf(p, 1.f - s, 1.f);
}

template <typename OUT> __device__ __forceinline__ void store4(OUT* p, const float (&x)[kV]) {
  store_raw<OUT, kV>(p, pack_as<OUT, kV>(x));
}

// Rows t0 - K .. t0 - 1 of sequence s (from row lo on; its initial state before).
template <typename IO, int K>
__device__ __forceinline__ void load_window(const ConvBwdArgs& a, int s, long long lo,
                                            long long t0, int c, float (&win)[K][kV]) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const long long t = t0 - K + i;
    Raw<IO, kV> v = zero_raw<IO, kV>();
    if (t >= lo)
      v = load_raw<IO, kV>((const IO*)a.x + t * a.x_stride + c);
    else if (a.init_state)
      v = load_raw<IO, kV>(
          (const IO*)a.init_state + ((long long)s * K + K - (lo - t)) * a.D + c);
    unpack_as<IO, kV>(v, win[i]);
  }
}

template <typename IO, typename OUT, int W, bool SILU>
__global__ void __launch_bounds__(32 * kGroups)
conv_bwd_kernel(ConvBwdArgs a, float* partial, long long row_blocks) {
  constexpr int K = W - 1;
  const int lane = threadIdx.x, group = threadIdx.y;
  const int c = ((int)blockIdx.y * 32 + lane) * kV;
  const bool on = c < a.D;
  const long long rows = a.cu_seqlens ? (long long)a.T : (long long)a.B * a.T;
  const IO* x = (const IO*)a.x + c;
  const IO* dy = (const IO*)a.d_out + c;

  float w[kV][W], bias[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[i][k] = on ? __ldg(a.weight + (long long)(c + i) * W + k) : 0.f;
    bias[i] = on && a.bias ? __ldg(a.bias + c + i) : 0.f;
  }

  if ((long long)blockIdx.x >= row_blocks) {
    // the initial state's gradient, one sequence per group
    const long long s = ((long long)blockIdx.x - row_blocks) * kGroups + group;
    if (s >= a.B || !on) return;
    long long lo, hi;
    seq_rows(a.cu_seqlens, (int)s, a.T, &lo, &hi);
    if (lo < 0 || hi < lo || hi > rows) {
      if (lane == 0) atomicOr(a.status, kDevBadSeqlens);
      return;
    }
    float win[K][kV], g[K][kV];
    load_window<IO, K>(a, (int)s, lo, lo, c, win);
#pragma unroll
    for (int i = 0; i < K; ++i) {
#pragma unroll
      for (int e = 0; e < kV; ++e) g[i][e] = 0.f;
      // a sequence shorter than the filter leaves rows of its initial state in the final one
      if (a.d_final_state && i >= hi - lo)
        unpack_as<float, kV>(load_raw<float, kV>(
                                 a.d_final_state + (s * K + i - (hi - lo)) * a.D + c),
                             g[i]);
    }
#pragma unroll
    for (int t = 0; t < K; ++t) {
      if (lo + t < hi) {
        float xv[kV], dv[kV];
        unpack_as<IO, kV>(load_raw<IO, kV>(x + (lo + t) * a.x_stride), xv);
        unpack_as<IO, kV>(load_raw<IO, kV>(dy + (lo + t) * a.D), dv);
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          float p = bias[e];
#pragma unroll
          for (int k = 0; k < K; ++k) p = fmaf(w[e][k], win[k][e], p);
          p = fmaf(w[e][K], xv[e], p);
          const float dp = dv[e] * d_act<SILU>(p);
          // row i of the state is t + K - i tokens before token t
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (i >= t) g[i][e] = fmaf(w[e][i - t], dp, g[i][e]);
#pragma unroll
          for (int k = 0; k + 1 < K; ++k) win[k][e] = win[k + 1][e];
          win[K - 1][e] = xv[e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < K; ++i) store4<float>(a.d_init_state + (s * K + i) * a.D + c, g[i]);
    return;
  }

  float dw[kV][W], db[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[i][k] = 0.f;
  }
  long long r = ((long long)blockIdx.x * kGroups + group) * kRun;
  const long long r1 = min(r + kRun, rows);
  int s = r < r1 ? seq_of_row(a.cu_seqlens, a.B, a.T, r) : 0;
  while (on && r < r1) {
    long long lo, hi;
    seq_rows(a.cu_seqlens, s, a.T, &lo, &hi);
    if (lo > r || hi > rows) {
      atomicOr(a.status, kDevBadSeqlens);
      break;
    }
    const long long end = min(hi, r1);
    if (end > r) {
      float win[K][kV], dpw[K][kV];
      load_window<IO, K>(a, s, lo, r, c, win);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < kV; ++e) dpw[k][e] = 0.f;
      for (long long t = r; t < end + K; t += kUnroll) {
        Raw<IO, kV> xr[kUnroll], dr[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const bool in = t + u < min(hi, end + K);
          xr[u] = in ? load_raw<IO, kV>(x + (t + u) * a.x_stride)
                     : zero_raw<IO, kV>();
          dr[u] = in ? load_raw<IO, kV>(dy + (t + u) * a.D)
                     : zero_raw<IO, kV>();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const long long row = t + u, q = row - K;
          float xv[kV], dv[kV], dx[kV];
          unpack_as<IO, kV>(xr[u], xv);
          unpack_as<IO, kV>(dr[u], dv);
          const bool mine = row < end;
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            float p = bias[e];
#pragma unroll
            for (int k = 0; k < K; ++k) p = fmaf(w[e][k], win[k][e], p);
            p = fmaf(w[e][K], xv[e], p);
            // rows behind the sequence have dy = 0; what they would multiply
            // must not turn a neighbour's infinity into a NaN
            const float dp = row < hi ? dv[e] * d_act<SILU>(p) : 0.f;
            if (mine) {
              db[e] += dp;
#pragma unroll
              for (int k = 0; k < K; ++k) dw[e][k] = fmaf(dp, win[k][e], dw[e][k]);
              dw[e][K] = fmaf(dp, xv[e], dw[e][K]);
            }
            float d = w[e][0] * dp;  // dp_{q+K}
#pragma unroll
            for (int k = 0; k < K; ++k) d = fmaf(w[e][K - k], dpw[k][e], d);  // dp_{q+k}
            dx[e] = d;
#pragma unroll
            for (int k = 0; k + 1 < K; ++k) {
              win[k][e] = win[k + 1][e];
              dpw[k][e] = dpw[k + 1][e];
            }
            win[K - 1][e] = xv[e];
            dpw[K - 1][e] = dp;
          }
          if (q >= r && q < end) {
            if (a.d_final_state && q >= hi - K) {
              float f[kV];
              unpack_as<float, kV>(
                  load_raw<float, kV>(
                      a.d_final_state + ((long long)s * K + q - (hi - K)) * a.D + c),
                  f);
#pragma unroll
              for (int e = 0; e < kV; ++e) dx[e] += f[e];
            }
            store4<OUT>((OUT*)a.dx + q * a.D + c, dx);
          }
        }
      }
      r = end;
    }
    if (++s >= a.B) {
      if (r < r1) atomicOr(a.status, kDevBadSeqlens);
      break;
    }
  }

  // the block's sums: [W + 1][128 channels] from the 8 groups
  __shared__ float red[kGroups][W + 1][32 * kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) red[group][k][lane * kV + e] = dw[e][k];
    red[group][W][lane * kV + e] = db[e];
  }
  __syncthreads();
  const int tid = group * 32 + lane;
  for (int i = tid; i < (W + 1) * 32 * kV; i += 32 * kGroups) {
    const int k = i / (32 * kV), ch = i % (32 * kV);
    const int d = (int)blockIdx.y * 32 * kV + ch;
    if (d >= a.D) continue;
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) sum += red[g][k][ch];
    partial[((long long)blockIdx.x * (W + 1) + k) * a.D + d] = sum;
  }
}

// d_weight[d][k] and d_bias[d] from the blocks' partials.
__global__ void __launch_bounds__(256)
conv_bwd_sum_kernel(const float* partial, long long blocks, int D, int W, float* dw, float* db) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)(W + 1) * D) return;
  const int k = (int)(i / D), d = (int)(i % D);
  const long long step = (long long)(W + 1) * D;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  long long b = 0;
  for (; b + 4 <= blocks; b += 4)
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += partial[(b + u) * step + i];
  for (; b < blocks; ++b) s[0] += partial[b * step + i];
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  if (k < W) dw[(long long)d * W + k] = sum;
  else if (db) db[d] = sum;
}

long long bwd_blocks(long long rows) { return (rows + kRun * kGroups - 1) / (kRun * kGroups); }

template <typename IO, typename OUT, int W, bool SILU>
cudaError_t bwd_typed(const ConvBwdArgs& a, float* partial, cudaStream_t stream) {
  const long long rows = a.cu_seqlens ? (long long)a.T : (long long)a.B * a.T;
  const long long blocks = bwd_blocks(rows);
  const long long states = a.d_init_state ? ((long long)a.B + kGroups - 1) / kGroups : 0;
  if (blocks + states > 0)
    conv_bwd_kernel<IO, OUT, W, SILU>
        <<<dim3((unsigned)(blocks + states), (unsigned)((a.D + 32 * kV - 1) / (32 * kV))),
           dim3(32, kGroups), 0, stream>>>(a, partial, blocks);
  const long long n = (long long)(W + 1) * a.D;
  conv_bwd_sum_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(
      partial, blocks, a.D, W, a.d_weight, a.d_bias);
  return cudaGetLastError();
}

template <typename IO, typename OUT>
cudaError_t bwd_io(const ConvBwdArgs& a, float* partial, cudaStream_t stream) {
  switch (a.W) {
    case 2:
      return a.silu ? bwd_typed<IO, OUT, 2, true>(a, partial, stream)
                    : bwd_typed<IO, OUT, 2, false>(a, partial, stream);
    case 3:
      return a.silu ? bwd_typed<IO, OUT, 3, true>(a, partial, stream)
                    : bwd_typed<IO, OUT, 3, false>(a, partial, stream);
    default:
      return a.silu ? bwd_typed<IO, OUT, 4, true>(a, partial, stream)
                    : bwd_typed<IO, OUT, 4, false>(a, partial, stream);
  }
}

}  // namespace

size_t conv_bwd_workspace(long long rows, int D, int W) {
  return (size_t)bwd_blocks(rows) * (size_t)(W + 1) * (size_t)D * 4;
}

cudaError_t launch_conv_bwd(const ConvBwdArgs& a, void* workspace, cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  if (a.fp32_io) return bwd_io<float, float>(a, partial, stream);
  if (a.fp32_out) return bwd_io<__nv_bfloat16, float>(a, partial, stream);
  return bwd_io<__nv_bfloat16, __nv_bfloat16>(a, partial, stream);
}

}  // namespace gla
