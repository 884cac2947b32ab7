// gla_scan_step.cu -- one token of the selective scan for N sequences.
//
//     delta = softplus(dt + dt_bias)
//     h'[d][n] = exp(delta a[d][n]) h[d][n] + delta u b[n]        (fp32 page)
//     y[d] = (sum_n c[n] h'[d][n] + skip[d] u) * silu(z)
//
// The step streams the state: 8 bytes per (channel, n) against four inputs and
// one output per channel, so HBM should bound it; with one sequence at a time
// instruction issue and the latency of tables and inputs did (every lane of a
// channel computing the same softplus: 266 instructions a warp per 8 channels, 118
// us at 1280 sequences of 2048 x 16).  So a block takes four sequences at a time:
// NS / 4 adjacent lanes own a channel, four states (16 bytes) of each sequence
// each, but one lane computes the softplus and the gate of one of the four
// sequences, and the lanes exchange them.  A block owns 1024 / NS channels and
// walks the groups of four; the page tables of all its sequences are read
// first, pages and inputs of the next two groups arrive by asynchronous copies.
#include "gla_scan.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;

constexpr int kSeqs = 4;            // sequences at a time
constexpr int kAhead = 2;           // groups of them in flight
constexpr int kRing = kAhead + 1;
constexpr int kMostGroups = 256;    // groups a block walks

template <typename IO, int NS> struct StepSmem {
  static constexpr int CT = kThreads / (NS / 4);  // channels per block
  float4 state[kRing][kSeqs][kThreads];           // each thread its own
  IO rows[kRing][kSeqs][3][CT];                   // u, dt, z
  float bc[kRing][kSeqs][2][NS];
  int2 pages[kMostGroups * kSeqs];                // read, written; -1: nothing to do
};

template <typename IO, typename OUT, int NS>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanStepArgs p) {
  constexpr int LPC = NS / 4;
  constexpr int OWN = LPC == 2 ? 2 : 1;  // sequences whose inputs a lane handles
  using S = StepSmem<IO, NS>;
  constexpr int CT = S::CT;
  extern __shared__ __align__(16) unsigned char smem[];
  S& s = *reinterpret_cast<S*>(smem);
  const int tid = threadIdx.x, q = tid % LPC, lc = tid / LPC;
  const int d0 = (int)blockIdx.x * CT;
  const bool on = d0 + lc < p.D;
  const int ch = on ? d0 + lc : 0;  // lanes past the end still join the exchanges
  // reduce4 leaves a lane with the sums of these sequences; the lane that holds
  // sequence i's inputs first, within the channel's lanes
  const int mine = LPC == 2 ? 2 * q : LPC == 4 ? q : q / (LPC / 4 > 0 ? LPC / 4 : 1);
  auto holder = [](int i) { return LPC == 2 ? i / 2 : LPC == 4 ? i : i * (LPC / 4); };
  const int quads = (p.N + kSeqs - 1) / kSeqs;
  const int groups = (quads - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;
  const long long page = (long long)p.D * NS;
  float* state = p.state + (long long)ch * NS + q * 4;
  // the row of sequence i of group j
  auto row_of = [&](int j, int i) { return (blockIdx.y + j * (int)gridDim.y) * kSeqs + i; };

  for (int x = tid; x < groups * kSeqs; x += kThreads) {
    const int n = row_of(x / kSeqs, x % kSeqs);
    int f = -1, t = -1;
    if (n < p.N) {
      f = t = n;
      if (p.slots != nullptr) {
        f = __ldg(p.slots + n);
        t = p.out_slots ? __ldg(p.out_slots + n) : f;
        if (f < 0 || t < 0) {
          f = t = -1;
        } else if (f >= p.num_slots || t >= p.num_slots) {
          if (blockIdx.x == 0) atomicOr(p.status, kDevBadSeqlens);
          f = t = -1;
        }
      }
    }
    s.pages[x] = make_int2(f, t);
  }
  __syncthreads();

  constexpr int kChunk = 16 / (int)sizeof(IO);            // channels of a 16-byte copy
  constexpr int kCopies = kSeqs * 3 * CT / kChunk;        // copies of a group's u, dt, z
  auto copy_group = [&](int j, int buf) {                 // always one group of copies
    if (j < groups) {
#pragma unroll
      for (int i = 0; i < kSeqs; ++i) {
        const int f = s.pages[j * kSeqs + i].x;
        if (f >= 0) cp_async16(&s.state[buf][i][tid], state + f * page);
      }
#pragma unroll
      for (int x0 = 0; x0 < kCopies; x0 += kThreads) {
        const int x = x0 + tid, c0 = x % (CT / kChunk) * kChunk, what = x / (CT / kChunk) % 3;
        const int i = x / (CT / kChunk) / 3;
        const int n = x < kCopies ? row_of(j, i) : p.N;
        const IO* from = (const IO*)(what == 0 ? p.u : what == 1 ? p.dt : p.z);
        const long long stride = what == 0 ? p.u_stride : what == 1 ? p.dt_stride : p.z_stride;
        if (n < p.N && d0 + c0 < p.D && from != nullptr)
          cp_async16(&s.rows[buf][i][what][c0], from + n * stride + d0 + c0);
      }
    }
    cp_commit();
  };
  // b and c (aligned to an element only): a group's elements through registers
  constexpr int kBC = (kSeqs * 2 * NS + kThreads - 1) / kThreads;
  IO bc[kBC];
  auto load_bc = [&](int j) {
#pragma unroll
    for (int e = 0; e < kBC; ++e) {
      const int x = tid + e * kThreads, n = x % NS, what = x / NS % 2, i = x / NS / 2;
      bc[e] = from_f32<IO>(0.f);
      if (i < kSeqs && j < groups && row_of(j, i) < p.N) {
        const long long row = row_of(j, i);
        bc[e] = what == 0 ? ((const IO*)p.b)[row * p.b_stride + n]
                          : ((const IO*)p.c)[row * p.c_stride + n];
      }
    }
  };
  auto store_bc = [&](int buf) {
#pragma unroll
    for (int e = 0; e < kBC; ++e) {
      const int x = tid + e * kThreads;
      if (x < kSeqs * 2 * NS) (&s.bc[buf][0][0][0])[x] = to_f32(bc[e]);
    }
  };

  load_bc(0);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) copy_group(i, i);
  store_bc(0);
  load_bc(1);
  float4 a = __ldg(reinterpret_cast<const float4*>(p.a + (long long)ch * NS) + q);
  a.x *= kLog2e; a.y *= kLog2e; a.z *= kLog2e; a.w *= kLog2e;
  const float bias = p.dt_bias ? __ldg(p.dt_bias + ch) : 0.f;
  const float skip = p.skip ? __ldg(p.skip + ch) : 0.f;

  int buf = 0;
  for (int j = 0; j < groups; ++j) {
    const int nxt = buf + 1 == kRing ? 0 : buf + 1;
    cp_wait<kAhead - 1>();
    __syncthreads();  // the group is there; everyone has left the buffer before it
    copy_group(j + kAhead, buf == 0 ? kRing - 1 : buf - 1);
    store_bc(nxt);
    load_bc(j + 2);
    float e[OWN], w[OWN], y[kSeqs];
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      e[k] = to_f32(s.rows[buf][mine + k][1][lc]) + bias;
      if (p.softplus) e[k] = softplus<sizeof(IO) == 4>(e[k]);
      w[k] = e[k] * to_f32(s.rows[buf][mine + k][0][lc]);
    }
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
      const float ei = __shfl_sync(0xffffffffu, e[LPC == 2 ? i & 1 : 0], holder(i), LPC);
      const float wi = __shfl_sync(0xffffffffu, w[LPC == 2 ? i & 1 : 0], holder(i), LPC);
      const int to = s.pages[j * kSeqs + i].y;
      y[i] = 0.f;
      if (to >= 0) {  // uniform over the block
        const float4 h = s.state[buf][i][tid];
        const float4 b = *reinterpret_cast<const float4*>(&s.bc[buf][i][0][q * 4]);
        const float4 c = *reinterpret_cast<const float4*>(&s.bc[buf][i][1][q * 4]);
        float4 x;
        const f32x2 d0 = decay2<sizeof(IO) == 4>(pack2(ei * a.x, ei * a.y));
        const f32x2 d1 = decay2<sizeof(IO) == 4>(pack2(ei * a.z, ei * a.w));
        x.x = fmaf(d0.x, h.x, wi * b.x);
        x.y = fmaf(d0.y, h.y, wi * b.y);
        x.z = fmaf(d1.x, h.z, wi * b.z);
        x.w = fmaf(d1.y, h.w, wi * b.w);
        if (on) __stcs(reinterpret_cast<float4*>(state + to * page), x);
        y[i] = fmaf(c.x, x.x, fmaf(c.y, x.y, fmaf(c.z, x.z, c.w * x.w)));
      }
    }
    int first;
    reduce4<LPC>(y, q, &first);
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      if (on && s.pages[j * kSeqs + mine + k].y >= 0 &&
          (LPC <= 4 || q % (LPC > 4 ? LPC / 4 : 1) == 0)) {
        float o = fmaf(skip, to_f32(s.rows[buf][mine + k][0][lc]), y[k]);
        if (p.z) o *= silu(to_f32(s.rows[buf][mine + k][2][lc]));
        ((OUT*)p.out)[(long long)row_of(j, mine + k) * p.D + ch] = from_f32<OUT>(o);
      }
    }
    buf = nxt;
  }
  cp_wait<0>();
}

template <typename IO, typename OUT, int NS>
cudaError_t launch_typed(const ScanStepArgs& a, cudaStream_t stream) {
  constexpr int CT = StepSmem<IO, NS>::CT, smem = (int)sizeof(StepSmem<IO, NS>);
  const int tiles = (a.D + CT - 1) / CT;
  // one wave of blocks, or two where each still walks eight groups (1280 sequences of
  // 2048 x 16: bf16 61.9 and 61.1 us, fp32 rows 67.8 and 64.0; 256 sequences 15.6 and
  // 17.8); no more than there are groups of sequences
  const long long quads = ((long long)a.N + kSeqs - 1) / kSeqs;
  long long groups = 3 * 152 / tiles;
  if (groups < 1) groups = 1;
  if (quads >= 16 * groups) groups *= 2;
  if (groups * kMostGroups < quads) groups = (quads + kMostGroups - 1) / kMostGroups;
  if (groups > quads) groups = quads;
  auto kernel = scan_step_kernel<IO, OUT, NS>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel, smem, done);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)tiles, (unsigned)groups), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename IO, typename OUT>
cudaError_t launch_io(const ScanStepArgs& a, cudaStream_t stream) {
  switch (a.NS) {
    case 8: return launch_typed<IO, OUT, 8>(a, stream);
    case 16: return launch_typed<IO, OUT, 16>(a, stream);
    case 32: return launch_typed<IO, OUT, 32>(a, stream);
    default: return launch_typed<IO, OUT, 64>(a, stream);
  }
}

}  // namespace

cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t stream) {
  if (a.fp32_io) return launch_io<float, float>(a, stream);
  if (a.fp32_out) return launch_io<__nv_bfloat16, float>(a, stream);
  return launch_io<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

}  // namespace gla
