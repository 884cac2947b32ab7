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
// run.  Its rows come through a ring of its own in shared memory, eight rows
// ahead: the bytes in flight that HBM needs (about 45 KB a SM) without registers
// or barriers.  65536 x 2048 bf16 rows: four rows ahead in registers 170 us, through
// the ring with windows that move a register a row 95 us, with windows that turn
// through the places of a group's four rows 92 us, in shorter runs 85 us: 93 % of copy
// bandwidth.
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kGroup = 4;   // rows of a group of copies
constexpr int kAhead = 2;   // groups in flight
constexpr int kRing = kAhead + 1;

template <typename IO> constexpr int conv_vec() { return 16 / (int)sizeof(IO); }

template <typename IO, typename OUT, int W, bool SILU>
__global__ void __launch_bounds__(128, 5)
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
    if (a.final_state == nullptr) {  // there is none: the offsets of some sequences
      const int on = min(a.D / V, (int)blockDim.x);  // threads that have channels
      if (blockIdx.y == 0)
        check_offsets(a.cu_seqlens, a.B, rows, (long long)s * on + threadIdx.x, a.B, a.status);
      return;
    }
    long long lo, hi;
    seq_rows(a.cu_seqlens, s, a.T, &lo, &hi);
    if (!bounds_ok(lo, hi, rows)) {
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

  constexpr int P = V / 2;
  __shared__ __align__(16) uint4 ring[kRing][kGroup][128];
  const long long r0 = (long long)blockIdx.x * run, r1 = min(r0 + run, rows);
  const int own = (int)(r1 - r0);      // rows are counted from r0 in what follows
  const IO* px = x + r0 * a.x_stride;  // the next row to copy
  int ahead = 0, put = 0;
  auto copy_group = [&]() {
    if (ahead + kGroup <= own) {
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        cp_async16(&ring[put][u][threadIdx.x], px);
        px += a.x_stride;
      }
    } else {
#pragma unroll 1
      for (int u = 0; u < kGroup && ahead + u < own; ++u) {
        cp_async16(&ring[put][u][threadIdx.x], px);
        px += a.x_stride;
      }
    }
    ahead += kGroup;
    cp_commit();
    put = put + 1 == kRing ? 0 : put + 1;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) copy_group();
  // (behind the first copies, which take longest)
  // two adjacent channels a register pair
  // the last four rows of x: row i of a group in place i, so that the windows of
  // a group's rows turn through fixed registers
  static_assert(kGroup == 4 && K < kGroup, "the rows before the current one and itself");
  f32x2 w[P][W], bias[P], xr[kGroup][P];
  {
    float f[V][W], b[V];
    load_filters<W, V>(a.weight + (long long)c * W, f);
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 v = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + c + i))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
      b[i] = v.x; b[i + 1] = v.y; b[i + 2] = v.z; b[i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[i][k] = pack2(f[2 * i][k], f[2 * i + 1][k]);
      bias[i] = pack2(b[2 * i], b[2 * i + 1]);
    }
  }
  OUT* out = (OUT*)a.out + r0 * a.D + c;
  // the sequence of row r0, and its window there
  int s = seq_of_row(a.cu_seqlens, a.B, a.T, r0);
  long long lo = 0, hi = 0;
  int end = 0;  // the sequence's rows in this run
  auto enter = [&](int r, int u) {  // row r, the u-th of its group; false: malformed offsets
    seq_rows(a.cu_seqlens, s, a.T, &lo, &hi);
    if (lo > r0 + r || hi > rows) return false;
    end = (int)max(min(hi - r0, (long long)own), 0ll);
    Raw<IO, V> v[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const long long t = r0 + r - K + i;
      v[i] = zero_raw<IO, V>();
      if (t >= lo) v[i] = load_raw<IO, V>(x + t * a.x_stride);
      else if (init) v[i] = load_raw<IO, V>(init + ((long long)s * K + K - (lo - t)) * a.D + c);
    }
#pragma unroll
    for (int p = 0; p < kGroup; ++p)
      if (p == u)
#pragma unroll
        for (int i = 0; i < K; ++i) unpack_pairs<IO, V>(v[i], xr[(p + kGroup - K + i) % kGroup]);
    return true;
  };
  int get = 0;
  auto take = [&](int u) {  // the u-th row of a group
    unpack_pairs<IO, V>(
        load_raw<IO, V>(reinterpret_cast<const IO*>(&ring[get][u][threadIdx.x])), xr[u]);
    float y[V];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      f32x2 p = bias[i];
#pragma unroll
      for (int k = 0; k < W; ++k) p = fma2(w[i][k], xr[(u + kGroup - K + k) % kGroup][i], p);
      if (SILU) p = mul2(p, sigmoid2(p));
      unpack2(p, &y[2 * i], &y[2 * i + 1]);
    }
    store_raw<OUT, V>(out, pack_as<OUT, V>(y));
    out += a.D;
  };
  bool ok = enter(0, 0);
  for (int row = 0; row < own && ok; row += kGroup) {
    copy_group();
    cp_wait<kAhead>();
    if (row + kGroup <= end) {  // inside a sequence
#pragma unroll
      for (int u = 0; u < kGroup; ++u) take(u);
    } else {
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        if (row + u < own && ok) {
          while (r0 + row + u >= hi && ok) {  // the next sequence that has a row
            ++s;
            ok = s < a.B && enter(row + u, u);
          }
          if (ok) take(u);
        }
      }
    }
    get = get + 1 == kRing ? 0 : get + 1;
  }
  if (!ok && threadIdx.x == 0) atomicOr(a.status, kDevBadSeqlens);
  cp_wait<0>();
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
  load_filters<W, V>(a.weight + (long long)c * W, w);
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 v = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + c + i))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    p[i] = v.x; p[i + 1] = v.y; p[i + 2] = v.z; p[i + 3] = v.w;
  }
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
  store_raw<OUT, V>((OUT*)a.out + n * a.D + c, pack_as<OUT, V>(p));
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
  // Runs of at most 32 rows, so that SMs that are ahead take more of them: 65536 x 2048
  // bf16 rows in one wave of five blocks a SM 100 us, in runs of 57 88 us, of 32 85 us, of
  // 19 87 us.  Shorter ones for one wave where the rows are fewer: 8192 rows in one
  // wave 15.7 us, in two 17.8 us.  At least 8 rows (a run's first W - 1 rows are read
  // twice).
  const long long share = (rows * gy + 5 * 152 - 1) / (5 * 152);
  const int run = share < 8 ? 8 : share > 32 ? 32 : (int)((share + kGroup - 1) / kGroup * kGroup);
  const long long blocks = (rows + run - 1) / run;
  // an in-place state is written by a launch of its own: its initial rows are
  // read by the first runs of the sequences
  const bool apart = a.final_state != nullptr && a.final_state == a.init_state;
  // where no block reads a sequence's offsets for its final state, blocks of their own
  // check them (in the row blocks the check slowed the loop: 65536 x 2048 bf16 rows 93 us
  // instead of 85)
  const int on = vecs < threads ? vecs : threads;
  const long long more = a.final_state ? (apart ? 0 : a.B) : a.cu_seqlens ? (a.B + on - 1ll) / on : 0;
  auto kernel = conv_fwd_kernel<IO, OUT, W, SILU>;
  if (blocks + more > 0)
    kernel<<<dim3((unsigned)(blocks + more), gy), threads, 0, stream>>>(a, run, blocks);
  if (apart) kernel<<<dim3((unsigned)a.B, gy), threads, 0, stream>>>(a, run, 0);
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
