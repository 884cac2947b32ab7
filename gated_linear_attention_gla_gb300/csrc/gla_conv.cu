// gla_conv.cu -- the short causal convolution in front of a selective scan:
// prompts (dense or packed), its gradients, and single tokens over a pool.
//
//     p_t[d] = bias[d] + sum_j weight[d][W - 1 - j] x_{t-j}[d],   y = p or silu(p)
//
// j = 0 .. W - 1, W = 2, 3 or 4, one filter per channel; rows in front of a
// sequence come from its initial state (its last W - 1 inputs), or are zero.
//
// The prompt form reads x once and writes y once (2 and 2 bytes an element in
// bf16 against ~10 instructions): HBM bounds it.  A thread owns 16 bytes of
// adjacent channels and walks a run of rows with the last W - 1 rows in
// registers, so that a row is read once but for the W - 1 rows in front of a
// run; four rows' loads are in flight before the first is used.
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kUnroll = 4;  // rows in flight per thread

template <typename IO> constexpr int conv_vec() { return 16 / (int)sizeof(IO); }

// The V channels' filters and biases.
template <int W, int V>
__device__ __forceinline__ void load_filter(const float* weight, const float* bias, int c,
                                            float (&w)[V][W], float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[i][k] = __ldg(weight + (long long)(c + i) * W + k);
    b[i] = bias ? __ldg(bias + c + i) : 0.f;
  }
}

template <typename IO, typename OUT, int W, bool SILU>
__global__ void __launch_bounds__(128)
conv_fwd_kernel(ConvArgs a, int run, long long row_blocks) {
  constexpr int V = conv_vec<IO>();
  constexpr int K = W - 1;
  const int c = ((int)blockIdx.y * (int)blockDim.x + (int)threadIdx.x) * V;
  if (c >= a.D) return;
  const IO* x = (const IO*)a.x + c;
  const IO* init = (const IO*)a.init_state;
  const long long rows = a.cu_seqlens ? (long long)a.T : (long long)a.B * a.T;

  if ((long long)blockIdx.x >= row_blocks) {
    // the final state of one sequence: its last W - 1 inputs.  Every row is
    // read before the first is written (the state may be updated in place).
    const int s = (int)((long long)blockIdx.x - row_blocks);
    long long lo, hi;
    seq_rows(a.cu_seqlens, s, a.T, &lo, &hi);
    if (lo < 0 || hi < lo || hi > rows) {
      if (threadIdx.x == 0) atomicOr(a.status, kDevBadSeqlens);
      return;
    }
    Raw<IO, V> r[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const long long t = hi - K + i;
      if (t >= lo) r[i] = load_raw<IO, V>(x + t * a.x_stride);
      else if (init)  // before the sequence: row K - (lo - t) of the initial state
        r[i] = load_raw<IO, V>(
            init + ((long long)s * K + K - (lo - t)) * a.D + c);
      else r[i] = zero_raw<IO, V>();
    }
    IO* fin = (IO*)a.final_state + (long long)s * K * a.D + c;
#pragma unroll
    for (int i = 0; i < K; ++i) store_raw<IO, V>(fin + (long long)i * a.D, r[i]);
    return;
  }

  float w[V][W], bias[V];
  load_filter<W, V>(a.weight, a.bias, c, w, bias);
  OUT* out = (OUT*)a.out + c;
  long long r = (long long)blockIdx.x * run;
  const long long r1 = min(r + run, rows);
  int s = seq_of_row(a.cu_seqlens, a.B, a.T, r);
  while (r < r1) {
    long long lo, hi;
    seq_rows(a.cu_seqlens, s, a.T, &lo, &hi);
    if (lo > r || hi > rows) {  // malformed offsets: this run stops
      if (threadIdx.x == 0) atomicOr(a.status, kDevBadSeqlens);
      return;
    }
    const long long end = min(hi, r1);
    if (end > r) {
      float win[K][V];
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const long long t = r - K + i;
        Raw<IO, V> v = zero_raw<IO, V>();
        if (t >= lo) v = load_raw<IO, V>(x + t * a.x_stride);
        else if (init)
          v = load_raw<IO, V>(
              init + ((long long)s * K + K - (lo - t)) * a.D + c);
        unpack_as<IO, V>(v, win[i]);
      }
      auto step = [&](const Raw<IO, V>& raw, long long row, bool in) {
        float xv[V], y[V];
        unpack_as<IO, V>(raw, xv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float p = bias[i];
#pragma unroll
          for (int k = 0; k < K; ++k) p = fmaf(w[i][k], win[k][i], p);
          p = fmaf(w[i][K], xv[i], p);
          y[i] = SILU ? silu(p) : p;
#pragma unroll
          for (int k = 0; k + 1 < K; ++k) win[k][i] = win[k + 1][i];
          win[K - 1][i] = xv[i];
        }
        if (!in) return;
        if constexpr (sizeof(OUT) * V > 16) {  // fp32 results of 8 bf16 channels
          float lo4[4], hi4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) { lo4[i] = y[i]; hi4[i] = y[i + V / 2]; }
          store_raw<OUT, 4>(out + row * a.D, pack_as<OUT, 4>(lo4));
          store_raw<OUT, 4>(out + row * a.D + 4, pack_as<OUT, 4>(hi4));
        } else {
          store_raw<OUT, V>(out + row * a.D, pack_as<OUT, V>(y));
        }
      };
      // (one loop for whole and partial groups: rows behind the sequence load
      // zeros and store nothing)
      for (; r < end; r += kUnroll) {
        Raw<IO, V> v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          v[u] = r + u < end ? load_raw<IO, V>(x + (r + u) * a.x_stride) : zero_raw<IO, V>();
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) step(v[u], r + u, r + u < end);
      }
      r = end;
    }
    if (++s >= a.B) {  // no sequence holds the rows that are left
      if (r < r1 && threadIdx.x == 0) atomicOr(a.status, kDevBadSeqlens);
      break;
    }
  }
}

// One token: the window is the page's W - 1 rows and x; the page written gets
// the window's last W - 1 rows.  Every read precedes the first write, so a row
// may read and write the same page.
template <typename IO, typename OUT, int W, bool SILU>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvStepArgs a) {
  constexpr int V = conv_vec<IO>();
  constexpr int K = W - 1;
  const int c = ((int)blockIdx.x * (int)blockDim.x + (int)threadIdx.x) * V;
  const long long n = blockIdx.y + (long long)blockIdx.z * gridDim.y;
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
  IO* pool = (IO*)a.state + c;
  const Raw<IO, V> xr = load_raw<IO, V>((const IO*)a.x + n * a.x_stride + c);
  Raw<IO, V> old[K];
#pragma unroll
  for (int i = 0; i < K; ++i)
    old[i] = load_raw<IO, V>(pool + (from * K + i) * a.D);
  float w[V][W], p[V];
  load_filter<W, V>(a.weight, a.bias, c, w, p);
  float xv[V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    unpack_as<IO, V>(old[k], xv);
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = fmaf(w[i][k], xv[i], p[i]);
  }
  unpack_as<IO, V>(xr, xv);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    p[i] = fmaf(w[i][K], xv[i], p[i]);
    if (SILU) p[i] = silu(p[i]);
  }
  OUT* out = (OUT*)a.out + n * a.D + c;
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = from_f32<OUT>(p[i]);
#pragma unroll
  for (int i = 0; i + 1 < K; ++i)
    store_raw<IO, V>(pool + (to * K + i) * a.D, old[i + 1]);
  store_raw<IO, V>(pool + (to * K + K - 1) * a.D, xr);
}

template <typename IO, typename OUT, int W, bool SILU>
cudaError_t fwd_typed(const ConvArgs& a, cudaStream_t stream) {
  constexpr int V = conv_vec<IO>();
  const int vecs = a.D / V;
  const int threads = vecs >= 128 ? 128 : (vecs + 31) / 32 * 32;
  const unsigned gy = (unsigned)((vecs + threads - 1) / threads);
  const long long rows = a.cu_seqlens ? (long long)a.T : (long long)a.B * a.T;
  const int run = 32;
  const long long blocks = (rows + run - 1) / run;
  const long long states = a.final_state ? a.B : 0;
  // an in-place state is written by a launch of its own: its initial rows are
  // read by the first runs of the sequences
  const bool apart = a.final_state != nullptr && a.final_state == a.init_state;
  if (blocks + (apart ? 0 : states) > 0)
    conv_fwd_kernel<IO, OUT, W, SILU>
        <<<dim3((unsigned)(blocks + (apart ? 0 : states)), gy), threads, 0, stream>>>(a, run,
                                                                                     blocks);
  if (apart && states > 0)
    conv_fwd_kernel<IO, OUT, W, SILU><<<dim3((unsigned)states, gy), threads, 0, stream>>>(a, run,
                                                                                         0);
  return cudaGetLastError();
}

template <typename IO, typename OUT, int W, bool SILU>
cudaError_t step_typed(const ConvStepArgs& a, cudaStream_t stream) {
  constexpr int V = conv_vec<IO>();
  const int vecs = a.D / V;
  const int threads = vecs >= 128 ? 128 : (vecs + 31) / 32 * 32;
  const unsigned ny = a.N < 32768 ? (unsigned)a.N : 32768u;
  const dim3 grid((unsigned)((vecs + threads - 1) / threads), ny, (unsigned)((a.N + ny - 1) / ny));
  conv_step_kernel<IO, OUT, W, SILU><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

#define GLA_CONV_BY_WIDTH(FN, IO, OUT)                                             \
  switch (a.W) {                                                                   \
    case 2: return a.silu ? FN<IO, OUT, 2, true>(a, stream) : FN<IO, OUT, 2, false>(a, stream); \
    case 3: return a.silu ? FN<IO, OUT, 3, true>(a, stream) : FN<IO, OUT, 3, false>(a, stream); \
    default: return a.silu ? FN<IO, OUT, 4, true>(a, stream) : FN<IO, OUT, 4, false>(a, stream); \
  }

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t stream) {
  if (a.fp32_io) { GLA_CONV_BY_WIDTH(fwd_typed, float, float) }
  if (a.fp32_out) { GLA_CONV_BY_WIDTH(fwd_typed, __nv_bfloat16, float) }
  GLA_CONV_BY_WIDTH(fwd_typed, __nv_bfloat16, __nv_bfloat16)
}

cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t stream) {
  if (a.fp32_io) { GLA_CONV_BY_WIDTH(step_typed, float, float) }
  if (a.fp32_out) { GLA_CONV_BY_WIDTH(step_typed, __nv_bfloat16, float) }
  GLA_CONV_BY_WIDTH(step_typed, __nv_bfloat16, __nv_bfloat16)
}

}  // namespace gla
