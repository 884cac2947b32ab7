// gla_recur_fwd.cuh -- the gated linear recurrence of a prompt.
//
//     log a = decay sigmoid(f) | log sigmoid(f);   m = sqrt(1 - a^2) | 1 - a
//     h_t = a h_{t-1} + m sigmoid(i) x;            y_t = h_t silu(z)
//
// gla_recur.cuh says how the token axis is split.  A warp's rows come through a
// tile of its own in shared memory (16-byte asynchronous copies; the next step's
// go out as soon as the rows are in registers).  First pass: gates, and the running
// map (P_t, H_t) of every token in registers; second pass, with the state in front
// of the run: h_t = P_t h + H_t.
// What takes the time: latency between dependent instructions, and 24 of 152 SMs have no block.  8192 x 2048 with
// three gates 39 us (4.3 TB/s; 68 % of the issue slots of 128 SMs), 20001 packed rows with two 86 us (3.8 TB/s;
// issue 56 %, DRAM 41 %, the cluster's exchange); fp32 rows 8192 x 2048 56 us (5.9 TB/s).
// The same kernel without its outputs (KEEP) writes the state in front of every
// kKeep tokens for the backward pass.
#pragma once

#include <type_traits>

#include "gla_recur.cuh"

namespace gla {
namespace recur {
namespace {

// A block's shape: tokens of a run, warps that compute (the exchange's comes on top), runs of
// a warp whose rows are in flight or in use.
template <int RUN, int WARPS, int STAGES, bool ALONE = false> struct Tile {
  static constexpr int kRun = RUN, kWarps = WARPS, kStages = STAGES;
  static constexpr bool kAlone = ALONE;  // for a cluster of one block
};
// Long runs spread the exchange of a cluster over more tokens and cost registers (16 warps of 128);
// where a block walks its sequence alone short ones with more warps are faster: 8192 x 2048
// 45 us by runs of 8, 40 us by runs of 4; 20001 packed rows in clusters of 4 92 and 134 us.  (Without the
// code for clusters 39.0 us, with it 40.4; 1 x 100 tokens x 512 by one block of long runs 4.4 us, by two of
// short ones 5.3.)
using LongRuns = Tile<8, 15, 2>;
using ShortRuns = Tile<4, 19, 3, true>;
using WideRuns = Tile<4, 15, 2>;  // fp32 rows
constexpr int kBlocks = 1;        // an SM

// DECAY, GATE, OUT: with decay, i, z.  STARTS: a group holds several sequences.  KEEP: see above.
template <typename T, typename TILE, bool DECAY, bool GATE, bool OUT, bool STARTS, bool KEEP>
__global__ void __launch_bounds__(32 * (TILE::kWarps + 1), kBlocks)
recur_kernel(RecurArgs a, Split p, float* kept, long long kept_rows) {
  after_previous();
  start_next();
  extern __shared__ __align__(16) unsigned char shared[];
  Maps& maps = *reinterpret_cast<Maps*>(shared);
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int kL = TILE::kRun, kStages = TILE::kStages;
  constexpr int kTile = kL * kChans;  // elements of a stream
  constexpr int kStreams = 2 + GATE + OUT;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = p.warps;
  const int rank = blockIdx.x % p.cluster;
  const long long unit = blockIdx.x / p.cluster, g = unit / p.cols;
  const int c0 = (int)(unit % p.cols) * kChans, c = c0 + 2 * lane;
  const bool on = c < a.D;
  long long lo, hi;
  group_rows(p, a.B, a.T, g, &lo, &hi);
  const long long reach = (long long)p.cluster * warps * kL;
  const long long steps = (hi - lo + reach - 1) / reach;
  auto init_of = [&](long long s) {
    return a.init_state && on ? *reinterpret_cast<const float2*>(a.init_state + s * a.D + c)
                              : both(0.f);
  };
  auto finish = [&](long long s, f32x2 h) {
    if (on) *reinterpret_cast<float2*>(a.final_state + s * a.D + c) = h;
  };
  // The initial state has been read by every block of the cluster before the first exchange, behind
  // which one of them may write the final state in its place (the store waits for the load).
  if (!STARTS && w == warps) maps.front[0][0][lane] = init_of(g);
  maps_init(maps, warps, p.cluster);

  Came came;
  if (w == warps) {
    f32x2 state = STARTS ? both(0.f) : maps.front[0][0][lane];
    state = TILE::kAlone || p.cluster == 1
                ? exchange_alone<STARTS>(maps, steps, warps, lane, state, a)
                : exchange<STARTS>(maps, steps, warps, rank, p.cluster, lane, state, a, came);
    if (!KEEP && !STARTS && a.final_state && rank == 0) finish(g, state);
  } else {
    T* const tiles = reinterpret_cast<T*>(shared + sizeof(Maps)) + w * kStages * kStreams * kTile;
    T* tile = tiles;  // of the run at hand
    const long long row0 = lo + ((long long)rank * warps + w) * kL;
    Stream<T, kL> streams[kStreams];
    streams[0].init(a.x, a.x_stride, row0, reach, c0, a.D, lane);
    streams[1].init(a.f, a.f_stride, row0, reach, c0, a.D, lane);
    if (GATE) streams[2].init(a.i, a.i_stride, row0, reach, c0, a.D, lane);
    if (OUT) streams[kStreams - 1].init(a.z, a.z_stride, row0, reach, c0, a.D, lane);
    auto fetch = [&](T* tile, long long r) {
      if (r < hi) {
        const int n = (int)(hi - r < kL ? hi - r : kL);
#pragma unroll
        for (int k = 0; k < kStreams; ++k) {
          streams[k].copy(tile + k * kTile, n, lane);
          streams[k].next();
        }
      }
      cp_commit();
    };
    for (int k = 0; k < kStages; ++k) fetch(tiles + k * kStreams * kTile, row0 + k * reach);

    f32x2 dec = both(0.f);
    if (DECAY && on) dec = decay_log2(*reinterpret_cast<const float2*>(a.decay + c));
    Seqs seqs(a.cu_seqlens, a.B, a.T);
    if (STARTS && a.cu_seqlens != nullptr) {
      if (c0 == 0)
        check_offsets(a.cu_seqlens, a.B, a.T, ((long long)rank * warps + w) * 32 + lane,
                      (long long)p.cluster * warps * 32, a.status);
      if (!KEEP && a.final_state)  // empty sequences hand their state through
        for (long long s = (long long)rank * warps + w; s < a.B; s += (long long)p.cluster * warps)
          if (__ldg(a.cu_seqlens + s) == __ldg(a.cu_seqlens + s + 1)) finish(s, init_of(s));
    }

    // whether every lane's decays are near enough to 1 for the shorter exponential
    const bool near = !DECAY || __all_sync(0xffffffffu, dec.x >= kNear && dec.y >= kNear);

    // A run between its two passes: token t's output is P front + H (with its output
    // gate in both), front being the state in front of the run.
    struct Run {
      f32x2 P[KEEP ? kL / kKeep : kL], H[KEEP ? kL / kKeep : kL];
      f32x2 Pe, He;  // the same for the state behind the last row of the run's first sequence
      long long r0;
      int n, s, fresh;  // rows; sequence of the first; first token that begins a sequence
      bool plain, ends; // a whole run inside one sequence; that sequence ends in it
    };
    auto first_pass = [&](Run& u, long long r0, long long step) {
      u.r0 = r0;
      u.n = r0 < hi ? (int)(hi - r0 < kL ? hi - r0 : kL) : 0;
      u.fresh = kL;
      f32x2 q = both(1.f), h = both(0.f);
      if (STARTS && u.n > 0) seqs.seek(r0);
      u.s = seqs.s;
      u.plain = u.n == kL && (!STARTS || (r0 != seqs.lo && r0 + kL <= seqs.hi));
      u.ends = STARTS && u.plain && r0 + kL == seqs.hi;
      cp_wait<kStages - 1>();
      __syncwarp();
      auto tokens = [&](auto straight, auto close) {
        constexpr bool PLAIN = decltype(straight)::value, NEAR = decltype(close)::value;
        int s = u.s;
        long long next = STARTS ? (r0 == seqs.lo ? r0 : seqs.hi) : 0;  // row of the next start
#pragma unroll
        for (int t = 0; t < kL; ++t) {
          f32x2 gate;
          if (PLAIN || t < u.n) {
            const f32x2 x = pair_at(tile + t * kChans, lane);
            const f32x2 f = pair_at(tile + kTile + t * kChans, lane);
            const f32x2 i = GATE ? pair_at(tile + 2 * kTile + t * kChans, lane) : both(0.f);
            const Gate gt = gates<EXACT, DECAY, GATE, false, NEAR>(f, i, dec, a.unit);
            const f32x2 b = mul2(GATE ? mul2(gt.m, gt.si) : gt.m, x);
            if (!PLAIN && STARTS && r0 + t == next) {
              while (s < a.B - 1 && r0 + t >= seqs.hi) {
                ++s;
                seq_rows(a.cu_seqlens, s, a.T, &seqs.lo, &seqs.hi);
              }
              seqs.s = s;
              next = seqs.hi;
              h = fma2(gt.a, init_of(s), b);
              q = both(0.f);
              if (u.fresh == kL) u.fresh = t;
            } else {
              h = fma2(gt.a, h, b);
              q = mul2(gt.a, q);
            }
            if (!PLAIN && STARTS && !KEEP && a.final_state && r0 + t + 1 == seqs.hi) {
              if (u.fresh < kL) {
                finish(s, h);
              } else {
                u.Pe = q;
                u.He = h;
                u.ends = true;
              }
            }
            if (OUT) {
              const f32x2 z = pair_at(tile + (kStreams - 1) * kTile + t * kChans, lane);
              f32x2 sz;
              sigmoids<EXACT>(z, &sz, nullptr);
              gate = mul2(z, sz);
            }
          }
          if (KEEP ? (t + 1) % kKeep == 0 : true) {
            u.P[KEEP ? t / kKeep : t] = OUT ? mul2(q, gate) : q;
            u.H[KEEP ? t / kKeep : t] = OUT ? mul2(h, gate) : h;
          }
        }
      };
      if (u.plain && near) tokens(std::true_type(), std::true_type());
      else if (u.plain) tokens(std::true_type(), std::false_type());
      else tokens(std::false_type(), std::false_type());
      if (STARTS && u.plain) {
        u.Pe = q;
        u.He = h;
      }
      const bool anew = STARTS && u.fresh < kL;
      give(maps, (int)step, w, lane,
           anew ? make_float4(-1.f, -1.f, h.x, h.y) : make_float4(q.x, q.y, h.x, h.y));
      fetch(tile, r0 + kStages * reach);  // (every lane has read the tile: give's __syncwarp)
      tile = tile == tiles + (kStages - 1) * kStreams * kTile ? tiles : tile + kStreams * kTile;
    };

    auto second_pass = [&](Run& u, long long step) {
      const f32x2 front = take(maps, (int)step, w, lane, a.status);
      if constexpr (KEEP) {
        // in front of tokens 0, kKeep, ... of the run
        float* to = kept + (g * kept_rows + (u.r0 - lo) / kKeep) * a.D + c;
#pragma unroll
        for (int t = 0; t < kL; t += kKeep) {
          if (t < u.n && on) {
            f32x2 v = front;
            if (t > 0) {
              const int k = t / kKeep - 1 < 0 ? 0 : t / kKeep - 1;
              v = STARTS && u.fresh < t ? u.H[k] : fma2(u.P[k], front, u.H[k]);
            }
            *reinterpret_cast<float2*>(to + (long long)(t / kKeep) * a.D) = v;
          }
        }
      } else {
        if (STARTS && u.ends && a.final_state) finish(u.s, fma2(u.Pe, front, u.He));
        const long long at = u.r0 * a.D + c;
        auto rows = [&](auto straight, auto* out) {
          constexpr bool PLAIN = decltype(straight)::value;
          using OT = std::remove_pointer_t<decltype(out)>;
#pragma unroll
          for (int t = 0; t < kL; ++t, out += a.D) {
            if (PLAIN || t < u.n) {
              f32x2 v = fma2(u.P[t], front, u.H[t]);
              if (!PLAIN && STARTS && t >= u.fresh) v = u.H[t];
              store_pair<OT>(out, v);
            }
          }
        };
        if (on) {
          if (a.fp32_out) {
            if (u.plain) rows(std::true_type(), (float*)a.out + at);
            else rows(std::false_type(), (float*)a.out + at);
          } else {
            if (u.plain) rows(std::true_type(), (__nv_bfloat16*)a.out + at);
            else rows(std::false_type(), (__nv_bfloat16*)a.out + at);
          }
        }
      }
    };

    // the second pass of a run behind the first pass of the next one
    Run even, odd;
    long long r0 = row0;
    for (long long step = 0; step < steps; step += 2) {
      first_pass(even, r0, step);
      if (step > 0) second_pass(odd, step - 1);
      r0 += reach;
      if (step + 1 < steps) {
        first_pass(odd, r0, step + 1);
        r0 += reach;
      }
      second_pass(even, step);
    }
    if (steps > 0 && steps % 2 == 0) second_pass(odd, steps - 1);
    cp_wait<0>();
  }
  if (!TILE::kAlone && p.cluster > 1) part(maps, w == warps, lane, rank, p.cluster, came);
}

template <typename T, typename TILE, bool DECAY, bool GATE, bool OUT, bool STARTS, bool KEEP>
cudaError_t run_tile(const RecurArgs& a, const Split& p, float* kept, long long kept_rows,
                     cudaStream_t stream) {
  constexpr int kWarpBytes =
      TILE::kStages * (2 + GATE + OUT) * TILE::kRun * kChans * (int)sizeof(T);
  auto kernel = recur_kernel<T, TILE, DECAY, GATE, OUT, STARTS, KEEP>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      allow_shared(kernel, (int)sizeof(Maps) + TILE::kWarps * kWarpBytes, done);
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
  return cudaLaunchKernelEx(&cfg, kernel, a, p, kept, kept_rows);
}

template <typename T, bool DECAY, bool GATE, bool OUT, bool KEEP>
cudaError_t run(const RecurArgs& a, float* kept, long long kept_rows, cudaStream_t stream) {
  const bool packed = a.cu_seqlens != nullptr;
  auto of = [&](auto tile) {
    using TILE = decltype(tile);
    return split(a.B, a.T, a.D, packed, TILE::kRun, TILE::kWarps, kBlocks);
  };
  using Usual = std::conditional_t<sizeof(T) == 4, WideRuns, LongRuns>;
  const Split p = of(Usual());
  if (p.spg != 1) return run_tile<T, Usual, DECAY, GATE, OUT, true, KEEP>(a, p, kept, kept_rows, stream);
  if constexpr (sizeof(T) == 2) {
    const Split alone = of(ShortRuns());
    if (p.cluster == 1 && alone.cluster == 1)
      return run_tile<T, ShortRuns, DECAY, GATE, OUT, false, KEEP>(a, alone, kept, kept_rows, stream);
  }
  return run_tile<T, Usual, DECAY, GATE, OUT, false, KEEP>(a, p, kept, kept_rows, stream);
}

template <typename T>
cudaError_t keep_typed(const RecurArgs& a, float* kept, long long kept_rows, cudaStream_t stream) {
  if (a.decay) return a.i ? run<T, true, true, false, true>(a, kept, kept_rows, stream)
                          : run<T, true, false, false, true>(a, kept, kept_rows, stream);
  return a.i ? run<T, false, true, false, true>(a, kept, kept_rows, stream)
             : run<T, false, false, false, true>(a, kept, kept_rows, stream);
}

template <typename T, bool DECAY> cudaError_t fwd_typed(const RecurArgs& a, cudaStream_t stream) {
  if (a.i) return a.z ? run<T, DECAY, true, true, false>(a, nullptr, 0, stream)
                      : run<T, DECAY, true, false, false>(a, nullptr, 0, stream);
  return a.z ? run<T, DECAY, false, true, false>(a, nullptr, 0, stream)
             : run<T, DECAY, false, false, false>(a, nullptr, 0, stream);
}

}  // namespace
}  // namespace recur
}  // namespace gla
