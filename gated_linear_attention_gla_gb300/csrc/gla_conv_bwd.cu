// gla_conv_bwd.cu -- the gradients of the short causal convolution.
//
// With p recomputed and dp_t = dy_t silu'(p_t) (or dy_t):
//     dx_t[d]        = sum_j weight[d][W - 1 - j] dp_{t+j}[d]      (t + j inside the sequence)
//     d_weight[d][k] = sum_t dp_t[d] x_{t-(W-1)+k}[d],   d_bias[d] = sum_t dp_t[d]
// The final state is a copy of the last W - 1 rows, so its gradient adds to
// theirs; the initial state's rows are rows in front of the sequence.
//
// One pass over x and dy: a thread owns 4 adjacent channels and a run of rows,
// with the last W - 1 rows of x and of dp in registers; dx of a row leaves W - 1
// rows later, so a run reads W - 1 rows past its end (for their dp only).  The
// rows come through a ring of the thread's own in shared memory, eight rows
// ahead.  The weight's gradient is summed in registers over the run, in shared
// memory over a block's 8 runs, and written as one fp32 partial per block; a
// second launch sums the partials in block order and forms the initial states'
// gradients.  No atomics: the same inputs give the same bits.
//
// Bound: HBM (6 bytes an element in bf16) for many rows, 65536 x 2048 in 139 us (86 % of
// copy bandwidth); 8192 x 2048 take 28 us, of which 12 are the start of the runs, the
// block sums and the second launch.  Rows loaded as they are needed 55 us, through the
// ring 38 us, without checks and moves inside a sequence 31 us.
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kV = 4;         // channels per thread
constexpr int kGroups = 8;    // runs per block
constexpr int kThreads = 32 * kGroups;
constexpr int kGroup = 4;     // rows of a group of copies
constexpr int kAhead = 2;     // groups in flight
constexpr int kRing = kAhead + 1;

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

// dp = dy act'(p) of two channels
template <bool SILU> __device__ __forceinline__ f32x2 d_pre(f32x2 dy, f32x2 p) {
  if (!SILU) return dy;
  const f32x2 s = sigmoid2(p);
  // s (1 + p (1 - s)) = s + s p (1 - s)
  const f32x2 sp = mul2(s, p);
  return mul2(dy, fma2(sp, fma2(s, both(-1.f), both(1.f)), s));
}

template <typename IO, typename OUT, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 2)
conv_bwd_kernel(ConvBwdArgs a, float* partial, int run) {
  start_next();
  constexpr int K = W - 1;
  const int lane = threadIdx.x, group = threadIdx.y;
  const int c = ((int)blockIdx.x * 32 + lane) * kV;
  const bool on = c < a.D;
  const long long rows = a.cu_seqlens ? (long long)a.T : (long long)a.B * a.T;
  const IO* x = (const IO*)a.x + c;
  const IO* dy = (const IO*)a.d_out + c;

  float w[kV][W] = {}, bias[kV] = {};
  if (on) {
    load_filters<W, kV>(a.weight + (long long)c * W, w);
    if (a.bias) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.bias + c));
      bias[0] = v.x; bias[1] = v.y; bias[2] = v.z; bias[3] = v.w;
    }
  }

  constexpr int P = kV / 2;  // two adjacent channels a register pair
  f32x2 w2[P][W], bias2[P], dw[P][W], db[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    bias2[i] = pack2(bias[2 * i], bias[2 * i + 1]);
    db[i] = f32x2{};
#pragma unroll
    for (int k = 0; k < W; ++k) {
      w2[i][k] = pack2(w[2 * i][k], w[2 * i + 1][k]);
      dw[i][k] = f32x2{};
    }
  }
  extern __shared__ __align__(16) unsigned char smem[];
  using R = Raw<IO, kV>;
  constexpr int kBytes = kV * (int)sizeof(IO);
  auto ring = reinterpret_cast<R (*)[kGroup][2][kThreads]>(smem);  // [kRing]: x, dy
  const int tid = group * 32 + lane;
  const long long r0 = ((long long)blockIdx.y * kGroups + group) * run;
  const long long r1 = min(r0 + run, rows), stop = min(r1 + K, rows);  // rows own, rows read
  if (on && r0 < r1) {
    // Rows are counted from r0 in what follows.
    const int own = (int)(r1 - r0), read = (int)(stop - r0);
    const IO* px = x + r0 * a.x_stride;
    const IO* pd = dy + r0 * a.D;
    int ahead = 0, put = 0, get = 0;
    auto copy_group = [&]() {
      if (ahead + kGroup <= read) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          cp_async<kBytes>(&ring[put][u][0][tid], px);
          cp_async<kBytes>(&ring[put][u][1][tid], pd);
          px += a.x_stride;
          pd += a.D;
        }
      } else {
#pragma unroll 1
        for (int u = 0; u < kGroup && ahead + u < read; ++u) {
          cp_async<kBytes>(&ring[put][u][0][tid], px);
          cp_async<kBytes>(&ring[put][u][1][tid], pd);
          px += a.x_stride;
          pd += a.D;
        }
      }
      ahead += kGroup;
      cp_commit();
      put = put + 1 == kRing ? 0 : put + 1;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) copy_group();

    // The last four rows of x and of dp: row i of a group in place i, so that the
    // windows of a group's rows turn through fixed registers.
    static_assert(K < kGroup, "the rows before the current one and itself");
    f32x2 xr[kGroup][P], dpr[kGroup][P];
    int s = seq_of_row(a.cu_seqlens, a.B, a.T, r0);
    long long lo = 0, hi = 0;
    int first = 0, end = 0;  // the sequence's rows in this run, and those read behind it
    auto enter = [&](int r, int u) {  // row r, the u-th of its group; false: malformed offsets
      seq_rows(a.cu_seqlens, s, a.T, &lo, &hi);
      if (lo > r0 + r || hi > rows) return false;
      first = r;
      end = (int)max(min(hi - r0, (long long)read), 0ll);
      float w0[K][kV];
      load_window<IO, K>(a, s, lo, r0 + r, c, w0);
#pragma unroll
      for (int x = 0; x < kGroup; ++x)
        if (x == u)
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) {
              xr[(x + kGroup - K + k) % kGroup][i] = pack2(w0[k][2 * i], w0[k][2 * i + 1]);
              dpr[(x + kGroup - K + k) % kGroup][i] = f32x2{};
            }
      return true;
    };
    // dx of the row K before the u-th of its group, whose dp is in dpr[u]
    auto sum_dp = [&](int u, f32x2 (&d)[P]) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        d[i] = mul2(w2[i][0], dpr[u][i]);
#pragma unroll
        for (int k = 0; k < K; ++k)
          d[i] = fma2(w2[i][K - k], dpr[(u + kGroup - K + k) % kGroup][i], d[i]);
      }
    };
    OUT* const out = (OUT*)a.dx + r0 * a.D + c;
    auto put_dx = [&](OUT* to, const f32x2 (&d)[P]) {
      float o[kV];
#pragma unroll
      for (int i = 0; i < P; ++i) unpack2(d[i], &o[2 * i], &o[2 * i + 1]);
      store4<OUT>(to, o);
    };
    // ... where that row is of this sequence and run
    auto emit = [&](int u, int q) {
      f32x2 d[P];
      sum_dp(u, d);
      if (q < first || q >= own) return;
      const long long from_end = r0 + q - (hi - K);
      if (a.d_final_state && from_end >= 0) {
        f32x2 f[P];
        unpack_pairs<float, kV>(
            load_raw<float, kV>(a.d_final_state + ((long long)s * K + from_end) * a.D + c), f);
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = add2(d[i], f[i]);
      }
      put_dx(out + (long long)q * a.D, d);
    };
    auto clear = [&](int u) {
#pragma unroll
      for (int i = 0; i < P; ++i) dpr[u][i] = f32x2{};
    };
    // The u-th row of a group: dp, and its terms of the weight's gradient.
    auto take = [&](int u, bool count) {
      f32x2 dv[P];
      unpack_pairs<IO, kV>(ring[get][u][0][tid], xr[u]);
      unpack_pairs<IO, kV>(ring[get][u][1][tid], dv);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        f32x2 p = bias2[i];
#pragma unroll
        for (int k = 0; k < W; ++k)
          p = fma2(w2[i][k], xr[(u + kGroup - K + k) % kGroup][i], p);
        dpr[u][i] = d_pre<SILU>(dv[i], p);
      }
      if (count) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          db[i] = add2(db[i], dpr[u][i]);
#pragma unroll
          for (int k = 0; k < W; ++k)
            dw[i][k] = fma2(dpr[u][i], xr[(u + kGroup - K + k) % kGroup][i], dw[i][k]);
        }
      }
    };

    bool ok = enter(0, 0), more = ok;
    int row = 0;
    OUT* to = out - (long long)K * a.D;  // dx of row - K
    while (more) {
      copy_group();
      cp_wait<kAhead>();
      if (row >= first + K && row + kGroup <= min(end, own)) {
        // inside a sequence and the run: no checks, no moves
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          take(u, true);
          f32x2 d[P];
          sum_dp(u, d);
          put_dx(to, d);
          to += a.D;
        }
        row += kGroup;
      } else {
        to += (long long)kGroup * a.D;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          while (more && r0 + row >= hi) {  // the sequence ends here
            // the K rows before this one, which no dp follows: turn the places on
            // and back again
#pragma unroll
            for (int k = 0; k < K; ++k) {
              clear((u + k) % kGroup);
              emit((u + k) % kGroup, row + k - K);
            }
            ++s;
            more = hi < r1;
            ok = !more || s < a.B;
            if (more) more = ok = ok && enter(row, u);
          }
          more = more && row < read;
          if (more) {
            take(u, row < own);
            emit(u, row - K);
            ++row;
          }
        }
      }
      get = get + 1 == kRing ? 0 : get + 1;
    }
    // (a run that ends inside a sequence has read K rows more: all its rows are out)
    if (!ok) atomicOr(a.status, kDevBadSeqlens);
    cp_wait<0>();
  }
  __syncthreads();  // the rings become the block's sums

  // the block's sums: [W + 1][128 channels] from the 8 groups
  auto red = reinterpret_cast<float (*)[W + 1][32 * kV]>(smem);  // [kGroups]
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float2 v;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      unpack2(dw[i][k], &v.x, &v.y);
      *reinterpret_cast<float2*>(&red[group][k][lane * kV + 2 * i]) = v;
    }
    unpack2(db[i], &v.x, &v.y);
    *reinterpret_cast<float2*>(&red[group][W][lane * kV + 2 * i]) = v;
  }
  __syncthreads();
  for (int i = tid; i < (W + 1) * 32 * kV; i += 32 * kGroups) {
    const int k = i / (32 * kV), ch = i % (32 * kV);
    const int d = (int)blockIdx.x * 32 * kV + ch;
    if (d >= a.D) continue;
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) sum += red[g][k][ch];
    partial[((long long)blockIdx.y * (W + 1) + k) * a.D + d] = sum;
  }
}

// The initial state's gradient of sequence s, four channels a thread.
template <typename IO, int W, bool SILU>
__device__ __forceinline__ void d_init_rows(const ConvBwdArgs& a, long long s, int c, bool first) {
  constexpr int K = W - 1;
  const long long rows = a.cu_seqlens ? (long long)a.T : (long long)a.B * a.T;
  const IO* x = (const IO*)a.x + c;
  const IO* dy = (const IO*)a.d_out + c;
  float w[kV][W], bias[kV] = {};
  load_filters<W, kV>(a.weight + (long long)c * W, w);
  if (a.bias) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(a.bias + c));
    bias[0] = v.x; bias[1] = v.y; bias[2] = v.z; bias[3] = v.w;
  }
  long long lo, hi;
  seq_rows(a.cu_seqlens, (int)s, a.T, &lo, &hi);
  if (!bounds_ok(lo, hi, rows)) {
    if (first) atomicOr(a.status, kDevBadSeqlens);
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
}

// d_weight[d][k] and d_bias[d] from the blocks' partials; in the blocks behind those, the
// initial states' gradients, which need nothing of the launch before (it has started,
// so all that precedes it is complete) and run beside it.
template <typename IO, int W, bool SILU>
__global__ void __launch_bounds__(kThreads)
conv_bwd_sum_kernel(ConvBwdArgs a, const float* partial, long long blocks, unsigned sum_blocks) {
  if (blockIdx.x >= sum_blocks) {
    const int tiles = (a.D + 32 * kV - 1) / (32 * kV);
    if (blocks == 0) after_previous();  // there was no launch before
    const long long n = (long long)(blockIdx.x - sum_blocks) * kGroups + threadIdx.x / 32;
    const int lane = threadIdx.x % 32, c = ((int)(n % tiles) * 32 + lane) * kV;
    if (n / tiles < a.B && c < a.D) d_init_rows<IO, W, SILU>(a, n / tiles, c, lane == 0);
    return;
  }
  const int D = a.D;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (blocks == 0) after_previous();
  if (a.cu_seqlens)  // (an input, as above)
    check_offsets(a.cu_seqlens, a.B, a.T, i, (long long)sum_blocks * blockDim.x, a.status);
  after_previous();
  if (i >= (long long)(W + 1) * D) return;
  const int k = (int)(i / D), d = (int)(i % D);
  const long long step = (long long)(W + 1) * D;
  float s[8] = {};
  long long b = 0;
  for (; b + 8 <= blocks; b += 8)
#pragma unroll
    for (int u = 0; u < 8; ++u) s[u] += partial[(b + u) * step + i];
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (b + u < blocks) s[u] += partial[(b + u) * step + i];
  const float sum = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  if (k < W) a.d_weight[(long long)d * W + k] = sum;
  else if (a.d_bias) a.d_bias[d] = sum;
}

// Rows per run: one wave of blocks (two a SM), at least 8 (W - 1 more are read).  A block's
// start and sums cost more than waves of runs would even out: 16384 x 2048 rows in
// one wave 46 us, in runs of at most 64 57 us, of 32 64 us.
int bwd_run(long long rows, int D) {
  const long long tiles = (D + 32 * kV - 1) / (32 * kV);
  const long long run = (rows * tiles + 2 * 152 * kGroups - 1) / (2 * 152 * kGroups);
  return run < 8 ? 8 : (int)run;
}
long long bwd_blocks(long long rows, int D) {
  const long long per = (long long)bwd_run(rows, D) * kGroups;
  return (rows + per - 1) / per;
}

template <typename IO, typename OUT, int W, bool SILU>
cudaError_t bwd_typed(const ConvBwdArgs& a, float* partial, cudaStream_t stream) {
  const long long rows = a.cu_seqlens ? (long long)a.T : (long long)a.B * a.T;
  const long long blocks = bwd_blocks(rows, a.D);
  constexpr int rings = kRing * kGroup * 2 * kThreads * kV * (int)sizeof(IO);
  constexpr int sums = kGroups * (W + 1) * 32 * kV * 4;
  constexpr int smem = rings > sums ? rings : sums;
  auto kernel = conv_bwd_kernel<IO, OUT, W, SILU>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel, smem, done);
  if (e != cudaSuccess) return e;
  const int tiles = (a.D + 32 * kV - 1) / (32 * kV);
  // (the tiles of 2^24 channels are too many for a grid's second dimension, the blocks
  // of a tile's rows are at most about two a SM)
  if (blocks > 0)
    kernel<<<dim3((unsigned)tiles, (unsigned)blocks), dim3(32, kGroups), smem, stream>>>(
        a, partial, bwd_run(rows, a.D));
  const cudaError_t main = cudaGetLastError();
  if (main != cudaSuccess) return main;
  const long long sum_blocks = ((long long)(W + 1) * a.D + kThreads - 1) / kThreads;
  const long long states = a.d_init_state ? ((long long)a.B * tiles + kGroups - 1) / kGroups : 0;
  return launch_after(conv_bwd_sum_kernel<IO, W, SILU>, dim3((unsigned)(sum_blocks + states)),
                      dim3(kThreads), 0, stream, a, partial, blocks, (unsigned)sum_blocks);
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
  return (size_t)bwd_blocks(rows, D) * (size_t)(W + 1) * (size_t)D * 4;
}

cudaError_t launch_conv_bwd(const ConvBwdArgs& a, void* workspace, cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  if (a.fp32_io) return bwd_io<float, float>(a, partial, stream);
  if (a.fp32_out) return bwd_io<__nv_bfloat16, float>(a, partial, stream);
  return bwd_io<__nv_bfloat16, __nv_bfloat16>(a, partial, stream);
}

}  // namespace gla
