// gla_recur.cu -- the gated linear recurrence: prompts, and single tokens.
//
//     log a = decay sigmoid(f) | log sigmoid(f);   m = sqrt(1 - a^2) | 1 - a
//     h_t = a h_{t-1} + m sigmoid(i) x;            y_t = h_t silu(z)
//
// gla_recur.cuh says how the token axis is split.  A warp's rows come through a
// tile of its own in shared memory (16-byte asynchronous copies; the next step's
// go out as soon as the rows are in registers).  First pass: gates, and the running
// map (P_t, H_t) of every token in registers; second pass, with the state in front
// of the run: h_t = P_t h + H_t.
// The same kernel without its outputs (KEEP) writes the state in front of every
// kKeep tokens for the backward pass.
#include "gla_recur.cuh"

namespace gla {
namespace recur {

Split split(int B, int T, int D, bool packed, int run, int most) {
  Split p;
  p.cols = (D + kChans - 1) / kChans;
  // short sequences share a group, so that a step's runs are filled
  p.spg = packed ? 0 : T >= 256 ? 1 : T > 0 ? (512 + T - 1) / T : 1;
  if (p.spg > B) p.spg = B;
  p.groups = packed ? 1 : ((long long)B + p.spg - 1) / (p.spg > 0 ? p.spg : 1);
  p.rows = packed ? T : (long long)p.spg * T;
  const long long units = (long long)p.cols * p.groups;
  // enough blocks for two an SM, while every block has tokens
  p.warps = most;
  p.cluster = 1;
  while (p.cluster < kMaxCluster && units * p.cluster * 2 <= 2 * 152 &&
         (long long)p.cluster * p.warps * run < p.rows)
    p.cluster *= 2;
  while (p.warps > 1 && (long long)(p.warps / 2) * p.cluster * run >= p.rows) p.warps /= 2;
  return p;
}

namespace {

constexpr int kL = 8;  // tokens of a run

template <typename T, typename OT, bool DECAY, bool STARTS, bool KEEP>
__global__ void __launch_bounds__(32 * kMaxWarps, 2)
recur_kernel(RecurArgs a, Split p, float* kept, long long kept_rows) {
  start_next();
  extern __shared__ __align__(16) unsigned char shared[];
  Maps& maps = *reinterpret_cast<Maps*>(shared);
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int kTile = kL * kChans;  // elements of a stream
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = p.warps;
  const int rank = blockIdx.x % p.cluster;
  const long long unit = blockIdx.x / p.cluster, g = unit / p.cols;
  const int c0 = (int)(unit % p.cols) * kChans, c = c0 + 2 * lane;
  const bool on = c < a.D;
  const bool has_i = a.i != nullptr, has_z = !KEEP && a.z != nullptr;
  T* tile = reinterpret_cast<T*>(shared + sizeof(Maps)) + w * 4 * kTile;
  long long lo, hi;
  group_rows(p, a.B, a.T, g, &lo, &hi);
  const long long reach = (long long)p.cluster * warps * kL;
  long long r0 = lo + ((long long)rank * warps + w) * kL;

  auto fetch = [&](long long r) {
    const int n = r < hi ? (int)(hi - r < kL ? hi - r : kL) : 0;
    copy_rows<T, kL>(tile, a.x, a.x_stride, r, n, c0, a.D, lane);
    copy_rows<T, kL>(tile + kTile, a.f, a.f_stride, r, n, c0, a.D, lane);
    if (has_i) copy_rows<T, kL>(tile + 2 * kTile, a.i, a.i_stride, r, n, c0, a.D, lane);
    if (has_z) copy_rows<T, kL>(tile + 3 * kTile, a.z, a.z_stride, r, n, c0, a.D, lane);
    cp_commit();
  };
  fetch(r0);

  f32x2 dec = both(0.f);
  if (DECAY && on) {
    const float2 v = *reinterpret_cast<const float2*>(a.decay + c);
    dec = make_float2(fminf(v.x, 0.f) * kLog2e, fminf(v.y, 0.f) * kLog2e);
  }
  auto init_of = [&](long long s) {
    return a.init_state && on ? *reinterpret_cast<const float2*>(a.init_state + s * a.D + c)
                              : both(0.f);
  };
  auto finish = [&](long long s, f32x2 h) {
    if (on) *reinterpret_cast<float2*>(a.final_state + s * a.D + c) = h;
  };
  Seqs seqs(a.cu_seqlens, a.B, a.T);
  f32x2 state = both(0.f);
  if (!STARTS) state = init_of(g);
  if (STARTS && a.cu_seqlens != nullptr) {
    if (c0 == 0)
      check_offsets(a.cu_seqlens, a.B, a.T, (long long)rank * blockDim.x + threadIdx.x,
                    (long long)p.cluster * blockDim.x, a.status);
    if (!KEEP && a.final_state)  // empty sequences hand their state through
      for (long long s = (long long)rank * warps + w; s < a.B; s += (long long)p.cluster * warps)
        if (__ldg(a.cu_seqlens + s) == __ldg(a.cu_seqlens + s + 1)) finish(s, init_of(s));
  }

  int turn = 0;
  for (long long base = lo; base < hi; base += reach, r0 += reach, turn ^= 1) {
    const int n = r0 < hi ? (int)(hi - r0 < kL ? hi - r0 : kL) : 0;
    f32x2 P[kL], H[kL];
    uint32_t zr[KEEP ? 1 : kL * sizeof(T) / 2];
    int fresh = kL;  // the first token that begins a sequence
    f32x2 q = both(1.f), h = both(0.f);
    if (STARTS && n > 0) seqs.seek(r0);
    int s = seqs.s;
    long long next = STARTS ? (r0 == seqs.lo ? r0 : seqs.hi) : 0;  // row of the next start
    cp_wait<0>();
    __syncwarp();
#pragma unroll
    for (int t = 0; t < kL; ++t) {
      if (t < n) {
        const f32x2 x = pair_at(tile + t * kChans, lane);
        const f32x2 f = pair_at(tile + kTile + t * kChans, lane);
        const f32x2 i = has_i ? pair_at(tile + 2 * kTile + t * kChans, lane) : both(0.f);
        if constexpr (!KEEP) {
          if (has_z) {
            if constexpr (sizeof(T) == 4) {
              const float2 z = pair_at(tile + 3 * kTile + t * kChans, lane);
              zr[2 * t] = __float_as_uint(z.x);
              zr[2 * t + 1] = __float_as_uint(z.y);
            } else {
              zr[t] = reinterpret_cast<const uint32_t*>(tile + 3 * kTile + t * kChans)[lane];
            }
          }
        }
        const Gate gt = gates<EXACT, DECAY, false>(f, i, dec, has_i, a.unit);
        const f32x2 b = mul2(mul2(gt.m, gt.si), x);
        if (STARTS && r0 + t == next) {
          while (s < a.B - 1 && r0 + t >= seqs.hi) {
            ++s;
            seq_rows(a.cu_seqlens, s, a.T, &seqs.lo, &seqs.hi);
          }
          seqs.s = s;
          next = seqs.hi;
          h = fma2(gt.a, init_of(s), b);
          q = both(0.f);
          if (fresh == kL) fresh = t;
        } else {
          h = fma2(gt.a, h, b);
          q = mul2(gt.a, q);
        }
      }
      if (!KEEP || (t + 1) % kKeep == 0) {
        P[t] = q;
        H[t] = h;
      }
    }
    __syncwarp();
    fetch(r0 + reach);
    const bool anew = STARTS && fresh < kL;
    const float4 mine = anew ? make_float4(-1.f, -1.f, h.x, h.y) : make_float4(q.x, q.y, h.x, h.y);
    const f32x2 front = exchange(maps, turn, mine, w, warps, rank, p.cluster, lane, &state);
    if constexpr (KEEP) {
      // in front of tokens 0, kKeep, ... of the run
      float* to = kept + (g * kept_rows + (r0 - lo) / kKeep) * a.D + c;
#pragma unroll
      for (int t = 0; t < kL; t += kKeep) {
        if (t < n && on) {
          f32x2 v = front;
          if (t > 0) v = STARTS && fresh < t ? H[t ? t - 1 : 0] : fma2(P[t ? t - 1 : 0], front, H[t ? t - 1 : 0]);
          *reinterpret_cast<float2*>(to + (long long)(t / kKeep) * a.D) = v;
        }
      }
    } else {
      int fs = s;
      long long end = 0;
      if (STARTS && n > 0 && a.final_state) {
        // the sequence of the run's first row, again
        if (anew) seqs.seek(r0);
        fs = seqs.s;
        end = seqs.hi;
      }
      OT* out = (OT*)a.out + r0 * a.D + c;
#pragma unroll
      for (int t = 0; t < kL; ++t) {
        if (t < n) {
          f32x2 v = fma2(P[t], front, H[t]);
          if (STARTS && t >= fresh) v = H[t];
          if (STARTS && a.final_state) {
            while (fs < a.B - 1 && r0 + t >= end) {
              ++fs;
              seq_rows(a.cu_seqlens, fs, a.T, &seqs.lo, &seqs.hi);
              seqs.s = fs;
              end = seqs.hi;
            }
            if (r0 + t + 1 == end) finish(fs, v);
          }
          if (has_z) {
            f32x2 z;
            if constexpr (sizeof(T) == 4)
              z = make_float2(__uint_as_float(zr[2 * t]), __uint_as_float(zr[2 * t + 1]));
            else
              z = widen(zr[t]);
            f32x2 sz, nz;
            sigmoids2<EXACT>(z, &sz, &nz);
            v = mul2(v, mul2(z, sz));
          }
          if (on) store_pair<OT>(out + (long long)t * a.D, v);
        }
      }
    }
  }
  cp_wait<0>();
  if (!KEEP && !STARTS && a.final_state && rank == 0 && w == 0) finish(g, state);
}

template <typename T, bool DECAY, bool KEEP, typename OT>
cudaError_t run(const RecurArgs& a, const Split& p, float* kept, long long kept_rows,
                cudaStream_t stream) {
  const int smem = (int)sizeof(Maps) + p.warps * 4 * kL * kChans * (int)sizeof(T);
  const long long blocks = (long long)p.cols * p.groups * p.cluster;
  auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
    cudaError_t e = allow_shared(kernel, (int)sizeof(Maps) + kMaxWarps * 4 * kL * kChans * (int)sizeof(T), done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(32 * p.warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, p, kept, kept_rows);
  };
  static std::atomic<uint64_t> d0{0}, d1{0};
  return p.spg == 1 ? go(recur_kernel<T, OT, DECAY, false, KEEP>, d0)
                    : go(recur_kernel<T, OT, DECAY, true, KEEP>, d1);
}

template <typename T, typename OT>
__global__ void __launch_bounds__(256) recur_step_kernel(RecurStepArgs a) {
  const long long n = (long long)blockIdx.z * gridDim.y + blockIdx.y;
  const int c = ((int)blockIdx.x * (int)blockDim.x + (int)threadIdx.x) * 4;
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
  constexpr bool EXACT = sizeof(T) == 4;
  f32x2 x[2], f[2], i[2] = {}, z[2] = {};
  unpack_pairs<T, 4>(load_raw<T, 4>((const T*)a.x + n * a.x_stride + c), x);
  unpack_pairs<T, 4>(load_raw<T, 4>((const T*)a.f + n * a.f_stride + c), f);
  if (a.i) unpack_pairs<T, 4>(load_raw<T, 4>((const T*)a.i + n * a.i_stride + c), i);
  if (a.z) unpack_pairs<T, 4>(load_raw<T, 4>((const T*)a.z + n * a.z_stride + c), z);
  float4 dec = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.decay) dec = __ldg(reinterpret_cast<const float4*>(a.decay + c));
  const float4 old = *reinterpret_cast<const float4*>(a.state + from * a.D + c);
  const f32x2 h0[2] = {make_float2(old.x, old.y), make_float2(old.z, old.w)};
  const f32x2 d[2] = {make_float2(fminf(dec.x, 0.f) * kLog2e, fminf(dec.y, 0.f) * kLog2e),
                      make_float2(fminf(dec.z, 0.f) * kLog2e, fminf(dec.w, 0.f) * kLog2e)};
  f32x2 h[2];
  float y[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Gate g = a.decay ? gates<EXACT, true, false>(f[k], i[k], d[k], a.i != nullptr, a.unit)
                           : gates<EXACT, false, false>(f[k], i[k], d[k], a.i != nullptr, a.unit);
    h[k] = fma2(g.a, h0[k], mul2(mul2(g.m, g.si), x[k]));
    f32x2 v = h[k];
    if (a.z) {
      f32x2 sz, nz;
      sigmoids2<EXACT>(z[k], &sz, &nz);
      v = mul2(v, mul2(z[k], sz));
    }
    y[2 * k] = v.x;
    y[2 * k + 1] = v.y;
  }
  *reinterpret_cast<float4*>(a.state + to * a.D + c) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
  store_raw<OT, 4>((OT*)a.out + n * a.D + c, pack_as<OT, 4>(y));
}

}  // namespace

cudaError_t launch_keep(const RecurArgs& a, const Split& p, float* kept, long long kept_rows,
                        cudaStream_t stream) {
  if (a.fp32_io)
    return a.decay ? run<float, true, true, float>(a, p, kept, kept_rows, stream)
                   : run<float, false, true, float>(a, p, kept, kept_rows, stream);
  return a.decay ? run<__nv_bfloat16, true, true, float>(a, p, kept, kept_rows, stream)
                 : run<__nv_bfloat16, false, true, float>(a, p, kept, kept_rows, stream);
}

}  // namespace recur

cudaError_t launch_recur_fwd(const RecurArgs& a, cudaStream_t stream) {
  using namespace recur;
  using bf16 = __nv_bfloat16;
  const Split p = split(a.B, a.T, a.D, a.cu_seqlens != nullptr, kL, kMaxWarps);
  if (a.fp32_io)
    return a.decay ? run<float, true, false, float>(a, p, nullptr, 0, stream)
                   : run<float, false, false, float>(a, p, nullptr, 0, stream);
  if (a.fp32_out)
    return a.decay ? run<bf16, true, false, float>(a, p, nullptr, 0, stream)
                   : run<bf16, false, false, float>(a, p, nullptr, 0, stream);
  return a.decay ? run<bf16, true, false, bf16>(a, p, nullptr, 0, stream)
                 : run<bf16, false, false, bf16>(a, p, nullptr, 0, stream);
}

cudaError_t launch_recur_step(const RecurStepArgs& a, cudaStream_t stream) {
  const int vecs = a.D / 4;
  const int threads = vecs >= 128 ? 128 : (vecs + 31) / 32 * 32;
  const unsigned ny = a.N < 32768 ? (unsigned)a.N : 32768u;
  const dim3 grid((unsigned)((vecs + threads - 1) / threads), ny, (unsigned)((a.N + ny - 1) / ny));
  using bf16 = __nv_bfloat16;
  if (a.fp32_io) recur::recur_step_kernel<float, float><<<grid, threads, 0, stream>>>(a);
  else if (a.fp32_out) recur::recur_step_kernel<bf16, float><<<grid, threads, 0, stream>>>(a);
  else recur::recur_step_kernel<bf16, bf16><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gla
