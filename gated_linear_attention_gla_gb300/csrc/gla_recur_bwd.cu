// gla_recur_bwd.cu -- the gradient of the gated linear recurrence, from its inputs alone.
// With e_t = dL/dh_t, s = sigmoid, and k = -dm / d(log a) = a^2 / m | a:
//     e_t = dy_t silu(z_t) + a_{t+1} e_{t+1}          (d_final behind the last token)
//     c_t = a h_{t-1} - k s(i) x,                      d(log a)_t = e_t c_t
//     dx = e m s(i),   di = e m x s(i) (1 - s(i)),     dz = dy h silu'(z)
//     df = e c log a (1 - s(f))  (without decay: e c (1 - s(f))),   d_decay = sum e c s(f)
//     d_init = a_0 e_0
// Two launches.  The forward kernel walks x, f and i once and keeps the state in
// front of every kKeep = 4 tokens; then the same split of the token axis
// (gla_recur.cuh) runs over e from the end.  A run is those 4 tokens: its states come again from the kept
// one, everything else that does not depend on e is reduced to factors of it in
// registers (each gradient is e times one number), and the map (Q_t, K_t) of e over the
// run is composed as in the forward.  d_decay: sums in registers over a thread's tokens, partials per
// block, summed in block order by a third launch.  No atomics.
#include "gla_recur.cuh"

namespace gla {
namespace recur {
namespace {

constexpr int kL = kKeep;   // tokens of a run
constexpr int kWarps = 8;   // of a block (128 registers a thread, two blocks an SM)

template <typename T, typename GT, bool DECAY, bool STARTS>
__global__ void __launch_bounds__(32 * kWarps, 2)
recur_bwd_kernel(RecurBwdArgs b, Split p, const float* kept, long long kept_rows, float* partial) {
  start_next();
  after_previous();
  extern __shared__ __align__(16) unsigned char shared[];
  Maps& maps = *reinterpret_cast<Maps*>(shared);
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int kTile = kL * kChans;
  const RecurArgs& a = b.f;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = p.warps;
  const int rank = blockIdx.x % p.cluster;
  const long long unit = blockIdx.x / p.cluster, g = unit / p.cols;
  const int c0 = (int)(unit % p.cols) * kChans, c = c0 + 2 * lane;
  const bool on = c < a.D;
  const bool has_i = a.i != nullptr, has_z = a.z != nullptr;
  // a warp's tile: five streams, then the kept state
  T* tile = reinterpret_cast<T*>(shared + sizeof(Maps) +
                                 w * (5 * kTile * (int)sizeof(T) + kChans * 4));
  float* front_h = reinterpret_cast<float*>(tile + 5 * kTile);
  long long lo, hi;
  group_rows(p, a.B, a.T, g, &lo, &hi);
  const long long runs = (hi - lo + kL - 1) / kL;
  const long long reach = (long long)p.cluster * warps;
  long long run = runs - 1 - ((long long)rank * warps + w);  // the runs from the end

  auto fetch = [&](long long u) {
    if (u >= 0) {
      const long long r = lo + u * kL;
      const int n = (int)(hi - r < kL ? hi - r : kL);
      copy_rows<T, kL>(tile, a.x, a.x_stride, r, n, c0, a.D, lane);
      copy_rows<T, kL>(tile + kTile, a.f, a.f_stride, r, n, c0, a.D, lane);
      if (has_i) copy_rows<T, kL>(tile + 2 * kTile, a.i, a.i_stride, r, n, c0, a.D, lane);
      if (has_z) copy_rows<T, kL>(tile + 3 * kTile, a.z, a.z_stride, r, n, c0, a.D, lane);
      copy_rows<T, kL>(tile + 4 * kTile, b.d_out, a.D, r, n, c0, a.D, lane);
      if (lane < 16 && c0 + 4 * lane < a.D)
        cp_async16(front_h + 4 * lane, kept + (g * kept_rows + u) * a.D + c0 + 4 * lane);
    }
    cp_commit();
  };
  fetch(run);

  f32x2 dec = both(0.f);
  if (DECAY && on) {
    const float2 v = *reinterpret_cast<const float2*>(a.decay + c);
    dec = make_float2(fminf(v.x, 0.f) * kLog2e, fminf(v.y, 0.f) * kLog2e);
  }
  auto init_of = [&](long long s) {
    return a.init_state && on ? *reinterpret_cast<const float2*>(a.init_state + s * a.D + c)
                              : both(0.f);
  };
  auto last_of = [&](long long s) {
    return b.d_final_state && on
               ? *reinterpret_cast<const float2*>(b.d_final_state + s * a.D + c)
               : both(0.f);
  };
  auto first = [&](long long s, f32x2 v) {
    if (on && b.d_init_state) *reinterpret_cast<float2*>(b.d_init_state + s * a.D + c) = v;
  };
  Seqs seqs(a.cu_seqlens, a.B, a.T);
  f32x2 state = both(0.f), sum = both(0.f);
  if (!STARTS) state = last_of(g);
  if (STARTS && a.cu_seqlens != nullptr) {
    if (c0 == 0)
      check_offsets(a.cu_seqlens, a.B, a.T, (long long)rank * blockDim.x + threadIdx.x,
                    (long long)p.cluster * blockDim.x, a.status);
    for (long long s = (long long)rank * warps + w; s < a.B; s += reach)
      if (__ldg(a.cu_seqlens + s) == __ldg(a.cu_seqlens + s + 1)) first(s, last_of(s));
  }

  int turn = 0;
  for (long long base = 0; base < runs; base += reach, run -= reach, turn ^= 1) {
    const long long r0 = lo + run * kL;
    const int n = run >= 0 ? (int)(hi - r0 < kL ? hi - r0 : kL) : 0;
    f32x2 Q[kL], K[kL], ca[kL], cx[kL], cf[kL], ci[kL], cd[kL];
    int seq[kL];
    unsigned starts = 0, lasts = 0;
    cp_wait<0>();
    __syncwarp();
    f32x2 h = both(0.f);
    if (n > 0) {
      h = pair_at(front_h, lane);
      if (STARTS) seqs.seek(r0);
      else if (run == 0) h = init_of(g);
    }
#pragma unroll
    for (int t = 0; t < kL; ++t) {
      if (t < n) {
        if (STARTS) {
          while (seqs.s < a.B - 1 && r0 + t >= seqs.hi) {
            ++seqs.s;
            seq_rows(a.cu_seqlens, seqs.s, a.T, &seqs.lo, &seqs.hi);
          }
          seq[t] = seqs.s;
          if (r0 + t == seqs.lo) {
            starts |= 1u << t;
            h = init_of(seqs.s);
          }
          if (r0 + t + 1 == seqs.hi) lasts |= 1u << t;
        }
        const f32x2 x = pair_at(tile + t * kChans, lane);
        const f32x2 f = pair_at(tile + kTile + t * kChans, lane);
        const f32x2 i = has_i ? pair_at(tile + 2 * kTile + t * kChans, lane) : both(0.f);
        f32x2 dy = pair_at(tile + 4 * kTile + t * kChans, lane);
        const Gate gt = gates<EXACT, DECAY, true>(f, i, dec, has_i, a.unit);
        const f32x2 sx = mul2(gt.si, x);
        // c = a h_{t-1} - k s(i) x
        const f32x2 ah = mul2(gt.a, h);
        const f32x2 cc = fma2(mul2(gt.k, both(-1.f)), sx, ah);
        h = fma2(gt.m, sx, ah);
        if (has_z) {
          const f32x2 z = pair_at(tile + 3 * kTile + t * kChans, lane);
          f32x2 sz, nz;
          sigmoids2<EXACT>(z, &sz, &nz);
          // silu' = s + s z (1 - s)
          const f32x2 gate = mul2(z, sz);
          const f32x2 dz = mul2(mul2(dy, h), fma2(gate, nz, sz));
          if (on) store_pair<GT>((GT*)b.dz + (r0 + t) * a.D + c, dz);
          dy = mul2(dy, gate);
        }
        K[t] = dy;
        ca[t] = gt.a;
        cx[t] = mul2(gt.m, gt.si);
        ci[t] = mul2(mul2(gt.m, sx), gt.ni);
        if (DECAY) {
          cd[t] = mul2(cc, gt.sf);
          cf[t] = mul2(mul2(cc, gt.nf), mul2(gt.l, both(kLn2)));
        } else {
          cf[t] = mul2(cc, gt.nf);
        }
      }
    }
    // the run's map of e from its end
    f32x2 q = both(1.f), e = both(0.f);
    int fresh = -1;  // the last token that ends a sequence
#pragma unroll
    for (int t = kL - 1; t >= 0; --t) {
      if (t < n) {
        if (STARTS && (lasts >> t & 1)) {
          q = both(0.f);
          e = last_of(seq[t]);
          if (fresh < 0) fresh = t;
        }
        Q[t] = q;
        K[t] = add2(K[t], e);
        e = mul2(ca[t], K[t]);
        q = mul2(ca[t], q);
      }
    }
    __syncwarp();
    fetch(run - reach);
    const float4 mine = STARTS && fresh >= 0 ? make_float4(-1.f, -1.f, e.x, e.y)
                                             : make_float4(q.x, q.y, e.x, e.y);
    const f32x2 behind = exchange(maps, turn, mine, w, warps, rank, p.cluster, lane, &state);
#pragma unroll
    for (int t = 0; t < kL; ++t) {
      if (t < n) {
        f32x2 v = fma2(Q[t], behind, K[t]);
        if (STARTS && t <= fresh) v = K[t];
        if (STARTS && (starts >> t & 1)) first(seq[t], mul2(ca[t], v));
        if (DECAY) sum = fma2(v, cd[t], sum);
        if (on) {
          const long long at = (r0 + t) * a.D + c;
          store_pair<GT>((GT*)b.dx + at, mul2(v, cx[t]));
          store_pair<GT>((GT*)b.df + at, mul2(v, cf[t]));
          if (has_i) store_pair<GT>((GT*)b.di + at, mul2(v, ci[t]));
        }
      }
    }
  }
  cp_wait<0>();
  if (!STARTS && rank == 0 && w == 0) first(g, state);
  if (DECAY && b.d_decay) {
    float2* part = reinterpret_cast<float2*>(shared + sizeof(Maps));
    __syncthreads();
    part[threadIdx.x] = sum;
    __syncthreads();
    if (w == 0 && on) {
      for (int k = 1; k < warps; ++k) sum = add2(sum, part[32 * k + lane]);
      *reinterpret_cast<float2*>(partial + (g * p.cluster + rank) * a.D + c) = sum;
    }
  }
}

// Sums the blocks' partials in block order: 32 channels a block.
__global__ void __launch_bounds__(1024)
decay_sum_kernel(float* d_decay, const float* partial, long long parts, int D) {
  after_previous();
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float t = 0.f;
  if (c < D)
    for (long long k = threadIdx.y; k < parts; k += 32) t += partial[k * D + c];
  part[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    for (int k = 1; k < 32; ++k) t += part[k][threadIdx.x];
    d_decay[c] = t;
  }
}

size_t kept_floats(const Split& p, int D) {
  const long long rows = (p.rows + kKeep - 1) / kKeep;
  return (size_t)(p.groups * rows * D + 63) / 64 * 64;
}

template <typename T, typename GT, bool DECAY>
cudaError_t run(const RecurBwdArgs& b, const Split& p, float* kept, long long kept_rows,
                float* partial, cudaStream_t stream) {
  const int per_warp = 5 * kL * kChans * (int)sizeof(T) + kChans * 4;
  auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
    cudaError_t e = allow_shared(kernel, (int)sizeof(Maps) + kWarps * per_warp, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.cols * p.groups * p.cluster));
    cfg.blockDim = dim3(32 * p.warps);
    cfg.dynamicSmemBytes = (int)sizeof(Maps) + p.warps * per_warp;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, b, p, (const float*)kept, kept_rows, partial);
  };
  static std::atomic<uint64_t> d0{0}, d1{0};
  return p.spg == 1 ? go(recur_bwd_kernel<T, GT, DECAY, false>, d0)
                    : go(recur_bwd_kernel<T, GT, DECAY, true>, d1);
}

}  // namespace
}  // namespace recur

size_t recur_bwd_workspace(int B, long long rows, int D, bool packed) {
  using namespace recur;
  if (B <= 0) return 0;
  const Split p = split(B, (int)(packed ? rows : rows / B), D, packed, kL, kWarps);
  return (kept_floats(p, D) + (size_t)p.groups * p.cluster * D) * 4;
}

cudaError_t launch_recur_bwd(const RecurBwdArgs& b, void* workspace, cudaStream_t stream) {
  using namespace recur;
  using bf16 = __nv_bfloat16;
  const RecurArgs& a = b.f;
  if (a.B == 0)  // no sequences, no rows
    return b.d_decay ? cudaMemsetAsync(b.d_decay, 0, (size_t)a.D * 4, stream) : cudaSuccess;
  const bool packed = a.cu_seqlens != nullptr;
  const Split keep = split(a.B, a.T, a.D, packed, 8, kMaxWarps);
  const Split p = split(a.B, a.T, a.D, packed, kL, kWarps);
  float* kept = static_cast<float*>(workspace);
  float* partial = kept + kept_floats(p, a.D);
  const long long kept_rows = (p.rows + kKeep - 1) / kKeep;
  cudaError_t e = launch_keep(a, keep, kept, kept_rows, stream);
  if (e != cudaSuccess) return e;
  if (a.fp32_io)
    e = a.decay ? run<float, float, true>(b, p, kept, kept_rows, partial, stream)
                : run<float, float, false>(b, p, kept, kept_rows, partial, stream);
  else if (a.fp32_out)
    e = a.decay ? run<bf16, float, true>(b, p, kept, kept_rows, partial, stream)
                : run<bf16, float, false>(b, p, kept, kept_rows, partial, stream);
  else
    e = a.decay ? run<bf16, bf16, true>(b, p, kept, kept_rows, partial, stream)
                : run<bf16, bf16, false>(b, p, kept, kept_rows, partial, stream);
  if (e != cudaSuccess || !b.d_decay) return e;
  return launch_after(decay_sum_kernel, dim3((a.D + 31) / 32), dim3(32, 32), 0, stream, b.d_decay,
                      (const float*)partial, p.groups * p.cluster, a.D);
}

}  // namespace gla
