// gla_recur_bwd.cuh -- the second launch of the gradient (gla_recur_bwd.cu): e from the end.
#pragma once

#include <type_traits>

#include "gla_recur.cuh"

namespace gla {
namespace recur {
namespace {

constexpr int kL = kKeep;  // tokens of a run
// Runs of a warp whose rows are in flight or in use (gradients of 8192 x 2048: one 107.6 us, two
// 103.8, three 103.5 and too much shared memory for fp32).
constexpr int kBwdStages = 2;

// DECAY, GATE, OUT: with decay, i, z.  STARTS: a group holds several sequences.
template <typename T, bool DECAY, bool GATE, bool OUT, bool STARTS>
__global__ void __launch_bounds__(32 * (kBwdWarps + 1), kBwdBlocks)
recur_bwd_kernel(RecurBwdArgs b, Split p, const float* kept, long long kept_rows, float* partial) {
  start_next();
  after_previous();
  extern __shared__ __align__(16) unsigned char shared[];
  Maps& maps = *reinterpret_cast<Maps*>(shared);
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int kTile = kL * kChans;
  constexpr int kStreams = 3 + GATE + OUT;
  const RecurArgs& a = b.f;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = p.warps;
  const int rank = blockIdx.x % p.cluster;
  const long long unit = blockIdx.x / p.cluster, g = unit / p.cols;
  const int c0 = (int)(unit % p.cols) * kChans, c = c0 + 2 * lane;
  const bool on = c < a.D;
  long long lo, hi;
  group_rows(p, a.B, a.T, g, &lo, &hi);
  const long long runs = (hi - lo + kL - 1) / kL;
  const long long reach = (long long)p.cluster * warps;
  const long long steps = (runs + reach - 1) / reach;
  f32x2 sum = both(0.f);  // of d_decay
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
  maps_init(maps, warps, p.cluster);

  Came came;
  if (w == warps) {
    f32x2 state = STARTS ? both(0.f) : last_of(g);
    state = p.cluster == 1
                ? exchange_alone<STARTS>(maps, steps, warps, lane, state, a)
                : exchange<STARTS>(maps, steps, warps, rank, p.cluster, lane, state, a, came);
    if (!STARTS && rank == 0) first(g, state);
  } else {
    // a warp's tiles, one for every stage: its streams (x, f, dy, i, z), then the kept state
    constexpr int kStage = kStreams * kTile + kChans * 4 / (int)sizeof(T);
    T* const tiles = reinterpret_cast<T*>(shared + sizeof(Maps)) + w * kBwdStages * kStage;
    long long run = runs - 1 - ((long long)rank * warps + w);  // the runs from the end

    Stream<T, kL> streams[kStreams];
    {
      const long long r = lo + run * kL, back = -reach * kL;
      streams[0].init(a.x, a.x_stride, r, back, c0, a.D, lane);
      streams[1].init(a.f, a.f_stride, r, back, c0, a.D, lane);
      streams[2].init(b.d_out, a.D, r, back, c0, a.D, lane);
      if (GATE) streams[3].init(a.i, a.i_stride, r, back, c0, a.D, lane);
      if (OUT) streams[kStreams - 1].init(a.z, a.z_stride, r, back, c0, a.D, lane);
    }
    auto fetch = [&](T* tile, long long u) {
      if (u >= 0) {
        const long long left = hi - lo - u * kL;
        const int n = (int)(left < kL ? left : kL);
#pragma unroll
        for (int k = 0; k < kStreams; ++k) {
          streams[k].copy(tile + k * kTile, n, lane);
          streams[k].next();
        }
        if (lane < 16 && c0 + 4 * lane < a.D)
          cp_async16(reinterpret_cast<float*>(tile + kStreams * kTile) + 4 * lane,
                     kept + (g * kept_rows + u) * a.D + c0 + 4 * lane);
      }
      cp_commit();
    };
    for (int k = 0; k < kBwdStages; ++k) fetch(tiles + k * kStage, run - k * reach);

    f32x2 dec = both(0.f);
    if (DECAY && on) dec = decay_log2(*reinterpret_cast<const float2*>(a.decay + c));
    const bool near = !DECAY || __all_sync(0xffffffffu, dec.x >= kNear && dec.y >= kNear);
    Seqs seqs(a.cu_seqlens, a.B, a.T);
    if (STARTS && a.cu_seqlens != nullptr) {
      if (c0 == 0)
        check_offsets(a.cu_seqlens, a.B, a.T, ((long long)rank * warps + w) * 32 + lane,
                      reach * 32, a.status);
      for (long long s = (long long)rank * warps + w; s < a.B; s += reach)
        if (__ldg(a.cu_seqlens + s) == __ldg(a.cu_seqlens + s + 1)) first(s, last_of(s));
    }
    // n (kL: all) rows of one gradient
    auto store = [&](void* to, long long at, int n, const f32x2 (&v)[kL]) {
      if (!on) return;
      if (a.fp32_out) {
        float* o = (float*)to + at;
#pragma unroll
        for (int t = 0; t < kL; ++t, o += a.D)
          if (t < n) store_pair<float>(o, v[t]);
      } else {
        __nv_bfloat16* o = (__nv_bfloat16*)to + at;
#pragma unroll
        for (int t = 0; t < kL; ++t, o += a.D)
          if (t < n) store_pair<__nv_bfloat16>(o, v[t]);
      }
    };

    int step = 0;
    T* tile = tiles;
    for (long long base = 0; base < runs; base += reach, run -= reach, ++step) {
      const long long r0 = lo + run * kL, at = r0 * a.D + c;
      const int n = run >= 0 ? (int)(hi - r0 < kL ? hi - r0 : kL) : 0;
      f32x2 Q[kL], K[kL], ca[kL], cx[kL], cf[kL], ci[kL], cd[kL], dz[kL];
      int seq[kL];
      unsigned starts = 0, lasts = 0;
      cp_wait<kBwdStages - 1>();
      __syncwarp();
      f32x2 h = both(0.f);
      bool plain = n == kL;
      if (n > 0) {
        h = pair_at(reinterpret_cast<const float*>(tile + kStreams * kTile), lane);
        if (STARTS) {
          seqs.seek(r0);
          plain = plain && r0 != seqs.lo && r0 + kL < seqs.hi;
        } else if (run == 0) {
          h = init_of(g);
        }
      }
      auto first_pass = [&](auto straight, auto close) {
        constexpr bool PLAIN = decltype(straight)::value, NEAR = decltype(close)::value;
#pragma unroll
        for (int t = 0; t < kL; ++t) {
          if (PLAIN || t < n) {
            if (!PLAIN && STARTS) {
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
            const f32x2 i = GATE ? pair_at(tile + 3 * kTile + t * kChans, lane) : both(0.f);
            f32x2 dy = pair_at(tile + 2 * kTile + t * kChans, lane);
            const Gate gt = gates<EXACT, DECAY, GATE, true, NEAR>(f, i, dec, a.unit);
            const f32x2 sx = GATE ? mul2(gt.si, x) : x;
            // c = a h_{t-1} - k s(i) x
            const f32x2 ah = mul2(gt.a, h);
            const f32x2 cc = fma2(mul2(gt.k, both(-1.f)), sx, ah);
            h = fma2(gt.m, sx, ah);
            if (OUT) {
              const f32x2 z = pair_at(tile + (kStreams - 1) * kTile + t * kChans, lane);
              f32x2 sz, nz;
              sigmoids<EXACT>(z, &sz, &nz);
              // silu' = s + s z (1 - s)
              const f32x2 gate = mul2(z, sz);
              dz[t] = mul2(mul2(dy, h), fma2(gate, nz, sz));
              dy = mul2(dy, gate);
            }
            K[t] = dy;
            ca[t] = gt.a;
            cx[t] = GATE ? mul2(gt.m, gt.si) : gt.m;
            if (GATE) ci[t] = mul2(mul2(gt.m, sx), gt.ni);
            if (DECAY) {
              cd[t] = mul2(cc, gt.sf);
              cf[t] = mul2(mul2(cc, gt.nf), mul2(gt.l, both(kLn2)));
            } else {
              cf[t] = mul2(cc, gt.nf);
            }
          }
        }
      };
      // the run's map of e from its end
      f32x2 q = both(1.f), e = both(0.f);
      int fresh = -1;  // the last token that ends a sequence
      if (plain) {
        if (near) first_pass(std::true_type(), std::true_type());
        else first_pass(std::true_type(), std::false_type());
#pragma unroll
        for (int t = kL - 1; t >= 0; --t) {
          Q[t] = q;
          K[t] = add2(K[t], e);
          e = mul2(ca[t], K[t]);
          q = mul2(ca[t], q);
        }
      } else {
        first_pass(std::false_type(), std::false_type());
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
      }
      const float4 mine = STARTS && fresh >= 0 ? make_float4(-1.f, -1.f, e.x, e.y)
                                               : make_float4(q.x, q.y, e.x, e.y);
      give(maps, step, w, lane, mine);
      fetch(tile, run - kBwdStages * reach);
      tile = tile == tiles + (kBwdStages - 1) * kStage ? tiles : tile + kStage;
      if (OUT) store(b.dz, at, n, dz);
      const f32x2 behind = take(maps, step, w, lane, a.status);
      f32x2 v[kL];
#pragma unroll
      for (int t = 0; t < kL; ++t) {
        if (t < n) {
          v[t] = fma2(Q[t], behind, K[t]);
          if (STARTS && t <= fresh) v[t] = K[t];
          if (STARTS && (starts >> t & 1)) first(seq[t], mul2(ca[t], v[t]));
          if (DECAY) sum = fma2(v[t], cd[t], sum);
          cx[t] = mul2(v[t], cx[t]);
          cf[t] = mul2(v[t], cf[t]);
          if (GATE) ci[t] = mul2(v[t], ci[t]);
        }
      }
      store(b.dx, at, n, cx);
      store(b.df, at, n, cf);
      if (GATE) store(b.di, at, n, ci);
    }
    cp_wait<0>();
  }
  if (p.cluster > 1) part(maps, w == warps, lane, rank, p.cluster, came);
  if (DECAY && b.d_decay) {
    float2* part = reinterpret_cast<float2*>(shared + sizeof(Maps));
    __syncthreads();
    if (w < warps) part[threadIdx.x] = sum;
    __syncthreads();
    if (w == 0 && on) {
      for (int k = 1; k < warps; ++k) sum = add2(sum, part[32 * k + lane]);
      // (a decay above 0 acts as 0 whatever its value)
      const float2 d = *reinterpret_cast<const float2*>(a.decay + c);
      sum = make_float2(d.x > 0.f ? 0.f : sum.x, d.y > 0.f ? 0.f : sum.y);
      *reinterpret_cast<float2*>(partial + (g * p.cluster + rank) * a.D + c) = sum;
    }
  }
}

template <typename T, bool DECAY, bool GATE, bool OUT>
cudaError_t run(const RecurBwdArgs& b, const Split& p, const float* kept, long long kept_rows,
                float* partial, cudaStream_t stream) {
  constexpr int kWarpBytes =
      kBwdStages * ((3 + GATE + OUT) * kL * kChans * (int)sizeof(T) + kChans * 4);
  auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
    cudaError_t e = allow_shared(kernel, (int)sizeof(Maps) + kBwdWarps * kWarpBytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.cols * p.groups * p.cluster));
    cfg.blockDim = dim3(32 * (p.warps + 1));
    cfg.dynamicSmemBytes = (int)sizeof(Maps) + p.warps * kWarpBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, b, p, kept, kept_rows, partial);
  };
  static std::atomic<uint64_t> d0{0}, d1{0};
  return p.spg == 1 ? go(recur_bwd_kernel<T, DECAY, GATE, OUT, false>, d0)
                    : go(recur_bwd_kernel<T, DECAY, GATE, OUT, true>, d1);
}

template <typename T, bool DECAY>
cudaError_t bwd_typed(const RecurBwdArgs& b, const Split& p, const float* kept,
                      long long kept_rows, float* partial, cudaStream_t stream) {
  if (b.f.i) return b.f.z ? run<T, DECAY, true, true>(b, p, kept, kept_rows, partial, stream)
                          : run<T, DECAY, true, false>(b, p, kept, kept_rows, partial, stream);
  return b.f.z ? run<T, DECAY, false, true>(b, p, kept, kept_rows, partial, stream)
               : run<T, DECAY, false, false>(b, p, kept, kept_rows, partial, stream);
}

}  // namespace
}  // namespace recur
}  // namespace gla
