// gla_recur.cuh -- what the kernels of the gated linear recurrence share: the gates of a
// token, the tiles of rows, and how the token axis is split.
//
// A recurrence h_t = a_t h_{t-1} + b_t over a run of tokens is the map
// h -> P h + H of its own (P the product of the a_t), and such maps compose. So
// the token axis is split three ways: a warp takes a run of consecutive tokens
// (its lanes two channels each), a block of `warps` warps consecutive runs, and
// the blocks of a thread-block cluster consecutive blocks of runs.  Each step of
// the loop covers cluster x warps runs: the warps reduce their runs to maps, the
// block composes its warps' (shared memory), the cluster's blocks send theirs to one
// another (distributed shared memory, counted by a barrier of the receiver), and every thread
// finishes its tokens from registers with the state in front of its run.  Every input is
// read once.
#pragma once

#include "gla_ssm.cuh"

namespace gla {
namespace recur {

constexpr int kChans = 64;     // channels of a block: two a lane
constexpr int kMaxWarps = 19;  // runs of a block
constexpr int kMaxCluster = 8; // (all that share a sequence's 64 channels: 1 x 65536 x 64 139 us, gradients 471;
                               // 1 x 32768 x 256 74 and 244; 3 x 20000 x 512 87 and 281)

// ---------------------------------------------------------------- the gates
// A token's values for a pair of channels.
struct Gate {
  f32x2 sf, nf;  // sigmoid(f), 1 - sigmoid(f)
  f32x2 si, ni;  // sigmoid(i), 1 - sigmoid(i)  (with i only)
  f32x2 l;       // log2 of the decay (with `decay` only)
  f32x2 a, m;    // decay, factor of the drive
  f32x2 k;       // -dm / d(log a)
};

// Sigmoids of a pair and, where `n` is asked for, 1 - sigmoid without cancellation.
// Four special-function instructions a pair: one reciprocal of the product of several
// denominators saves two of them but costs ten others, and it is issue slots
// that bound these kernels (8192 x 2048 with three gates: 68 us with it, 43 us without, together
// with the square root below and the exchange by a warp of its own).
// 1 - s = e s with e = exp(-v).  From e = 2^126 on the reciprocal is subnormal and flushed, so that s is 0,
// and where e is infinite the product is NaN, which the minimum turns into 1.  Next to a factor s the
// zero is as good (and a NaN of v stays one in s).  ALONE: 1 - s is used without one (1 - a of the
// gate itself as decay), and is 1 where s is 0: s is 0 or at least 2^-126, so 1 - 2^126 s is 1 there
// and at most 0 elsewhere, and the larger of it and e s is 1 - s.  (For every 1 - s of the gradients
// of 8192 x 2048 that would cost 107.4 us for 103.9.)
// EXACT (fp32 rows): from e = exp(-|v|) with its argument's rounding taken back.
template <bool EXACT, bool ALONE = false>
__device__ __forceinline__ void sigmoids(f32x2 v, f32x2* s, f32x2* n) {
  if (EXACT) {
    const f32x2 e = exp_neg_abs2<true>(v), d = add2(e, both(1.f));
    const f32x2 q = make_float2(rcp(d.x), rcp(d.y)), p = mul2(e, q);
    *s = make_float2(v.x < 0.f ? p.x : q.x, v.y < 0.f ? p.y : q.y);
    if (n) *n = make_float2(v.x < 0.f ? q.x : p.x, v.y < 0.f ? q.y : p.y);
  } else {
    const f32x2 e = ex2x2(mul2(v, both(-kLog2e))), d = add2(e, both(1.f));
    *s = make_float2(rcp(d.x), rcp(d.y));
    if (n) {
      const f32x2 p = mul2(e, *s);
      if (ALONE) {
        const f32x2 shut = fma2(*s, both(-8.5070592e37f), both(1.f));  // 1 - 2^126 s
        *n = make_float2(fmaxf(p.x, shut.x), fmaxf(p.y, shut.y));
      } else {
        *n = make_float2(fminf(p.x, 1.f), fminf(p.y, 1.f));
      }
    }
  }
}

// 2^l and 1 - 2^l of l in [-126, 0] without the special-function unit and without
// cancellation near l = 0: l = k + r with |r| <= 1/2, (2^r - 1) / r by a
// polynomial of degree 5 (least maximal relative error there, by exchange of its
// extrema: 1.1e-8), 2^k in the exponent.  1 - a^2 = (1 - a)(2 - (1 - a))
// then keeps its relative accuracy for decays of 0.9999.
__device__ __forceinline__ void exp2m1(f32x2 l, f32x2* a, f32x2* u) {
  const f32x2 t = add2(l, both(12582912.f));  // its low bits: k
  const f32x2 r = fma2(add2(t, both(-12582912.f)), both(-1.f), l);
  f32x2 p = fma2(both(1.54035122e-4f), r, both(1.33907353e-3f));
  p = fma2(p, r, both(9.61823761e-3f));
  p = fma2(p, r, both(5.55035733e-2f));
  p = fma2(p, r, both(0.240226492f));
  p = fma2(p, r, both(0.693147182f));
  p = mul2(p, r);
  const f32x2 s = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                              __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));
  const f32x2 q = mul2(s, p);
  *a = add2(s, q);
  *u = fma2(q, both(-1.f), fma2(s, both(-1.f), both(1.f)));
}

// The same for l in [-2, 0] (kNear) without taking k apart: a polynomial of degree 6 over
// that range, off by 2.2e-8 of 2^l - 1.  A third of the instructions.
// (8192 x 2048 with one channel of every 64 below kNear, which takes the other for all of the warp:
// 38.9 -> 41.6 us, gradients 102.5 -> 108.8.)
constexpr float kNear = -2.f;
__device__ __forceinline__ void exp2m1_near(f32x2 l, f32x2* a, f32x2* u) {
  f32x2 p = fma2(both(-8.35481114e-6f), l, both(-1.36740666e-4f));
  p = fma2(p, l, both(-1.3104945e-3f));
  p = fma2(p, l, both(-9.60214809e-3f));
  p = fma2(p, l, both(-5.54986782e-2f));
  p = fma2(p, l, both(-0.240225807f));
  p = fma2(p, l, both(-0.693147182f));
  *u = mul2(p, l);
  *a = fma2(*u, both(-1.f), both(1.f));
}

// 0 where v is below the smallest normal number, as the square root of such a v is in sqrt_of
__device__ __forceinline__ float rsqrt_or_0(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return v < 1.17549435e-38f ? 0.f : r;
}
__device__ __forceinline__ float sqrt_of(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {  // a NaN stays one
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
// log2 of the decay at s(f) = 1 from the parameter (above 0 it counts as 0, a NaN stays one)
__device__ __forceinline__ f32x2 decay_log2(float2 v) {
  return make_float2((v.x > 0.f ? 0.f : v.x) * kLog2e, (v.y > 0.f ? 0.f : v.y) * kLog2e);
}

// `c`: decay log2(e) of the pair (DECAY); NEAR: it is at least kNear
template <bool EXACT, bool DECAY, bool GATE, bool BWD, bool NEAR>
__device__ __forceinline__ Gate gates(f32x2 f, f32x2 i, f32x2 c, bool unit) {
  Gate g;
  sigmoids<EXACT, !DECAY>(f, &g.sf, BWD || !DECAY ? &g.nf : nullptr);
  if (GATE) sigmoids<EXACT>(i, &g.si, BWD ? &g.ni : nullptr);
  f32x2 u;  // 1 - a
  if (DECAY) {
    g.l = mul2(c, g.sf);
    if (NEAR) {
      exp2m1_near(g.l, &g.a, &u);
    } else {
      g.l = make_float2(max_nan(g.l.x, -126.f), max_nan(g.l.y, -126.f));
      exp2m1(g.l, &g.a, &u);
    }
  } else {
    g.a = g.sf;
    u = g.nf;
  }
  // 1 - a^2 = u (2 - u).  Both factors are computed: a branch would part the tokens of a
  // run, whose latencies hide one another.
  if (BWD) {
    const f32x2 v = mul2(u, fma2(u, both(-1.f), both(2.f)));
    const f32x2 rs = make_float2(rsqrt_or_0(v.x), rsqrt_or_0(v.y));
    const f32x2 m = mul2(v, rs), k = mul2(mul2(g.a, g.a), rs);
    g.m = make_float2(unit ? m.x : u.x, unit ? m.y : u.y);
    g.k = make_float2(unit ? k.x : g.a.x, unit ? k.y : g.a.y);
  } else {
    const f32x2 v = mul2(u, fma2(u, both(-1.f), both(2.f)));
    g.m = make_float2(unit ? sqrt_of(v.x) : u.x, unit ? sqrt_of(v.y) : u.y);
  }
  return g;
}

// ---------------------------------------------------------------- rows in shared memory
// The pair at a lane's channels of one row of a tile.
template <typename T> __device__ __forceinline__ f32x2 pair_at(const T* row, int lane);
template <> __device__ __forceinline__ f32x2 pair_at<float>(const float* row, int lane) {
  return reinterpret_cast<const float2*>(row)[lane];
}
__device__ __forceinline__ f32x2 widen(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ f32x2 pair_at<__nv_bfloat16>(const __nv_bfloat16* row, int lane) {
  return widen(reinterpret_cast<const uint32_t*>(row)[lane]);
}

// A warp's asynchronous copies of runs of L rows of one stream: the lane's place in the
// first row, moved on from run to run (address arithmetic is a sixth of the work
// otherwise).
template <typename T, int L> struct Stream {
  static constexpr int kE = 16 / (int)sizeof(T), kPer = kChans / kE, kRows = 32 / kPer;
  const T* at;
  long long hop;   // elements between the lane's rows
  long long step;  // elements between the warp's runs
  int place;       // the lane's element of the tile
  bool on;         // the lane's channels exist
  __device__ __forceinline__ void init(const void* src, long long stride, long long row,
                                       long long rows_step, int c0, int D, int lane) {
    const int c = lane % kPer * kE;
    on = c0 + c < D;
    at = (const T*)src + (row + lane / kPer) * stride + c0 + c;
    hop = stride * kRows;
    step = stride * rows_step;
    place = lane / kPer * kChans + c;
  }
  // Rows [FROM, TO) of n at the current place.
  template <int FROM = 0, int TO = L>
  __device__ __forceinline__ void copy(T* tile, int n, int lane) const {
    static_assert(FROM % kRows == 0 && TO % kRows == 0, "whole groups of rows");
    const T* p = at + FROM / kRows * hop;
    if (!on) return;
    if (n >= TO) {
#pragma unroll
      for (int k = FROM; k < TO; k += kRows, p += hop) cp_async16(tile + place + k * kChans, p);
    } else {
#pragma unroll
      for (int k = FROM; k < TO; k += kRows, p += hop)
        if (k + lane / kPer < n) cp_async16(tile + place + k * kChans, p);
    }
  }
  __device__ __forceinline__ void next() { at += step; }
};

template <typename OT>
__device__ __forceinline__ void store_pair(OT* p, f32x2 v) {
  const float x[2] = {v.x, v.y};
  store_raw<OT, 2>(p, pack_as<OT, 2>(x));
}

// ---------------------------------------------------------------- composition
// A run's map of a lane's two channels (P, P, H, H).  STARTS: sequences may begin inside;
// P < 0 says that one does, so that nothing in front of it is multiplied,
// infinities included.
template <bool STARTS> __device__ __forceinline__ f32x2 apply(float4 map, f32x2 h) {
  const f32x2 v = fma2(make_float2(map.x, map.y), h, make_float2(map.z, map.w));
  if (!STARTS) return v;
  return make_float2(map.x < 0.f ? map.z : v.x, map.x < 0.f ? map.w : v.y);
}
// `next` after `map`
template <bool STARTS> __device__ __forceinline__ float4 compose(float4 map, float4 next) {
  f32x2 p = mul2(make_float2(map.x, map.y), make_float2(next.x, next.y));
  const f32x2 h = apply<STARTS>(next, make_float2(map.z, map.w));
  if (STARTS && (next.x < 0.f || map.x < 0.f)) p = both(-1.f);
  return make_float4(p.x, p.y, h.x, h.y);
}

// What a block's warps exchange, for two steps in turn: their maps, the maps of the
// cluster's blocks, and the state in front of each warp's run.  The block has a warp
// for the exchange beside the `warps` that compute: those hand a run's map over and
// work on their next run before they need the state in front of the one before, so that the
// latency of the exchange (a microsecond across a cluster) is not theirs.
struct Maps {
  float4 warp[2][kMaxWarps][32];
  float4 block[2][kMaxCluster][32];
  f32x2 front[2][kMaxWarps][32];
  uint64_t given[2];  // the warps' maps of a step are there
  uint64_t full[2];   // counts the bytes of block[turn]
  uint64_t ready[2];  // front[turn] is there
  int given_up;       // a wait of the block ran out
  uint32_t told[kMaxCluster];  // how many steps each block's exchange has sent, + kGaveUp
};
constexpr uint32_t kGaveUp = 0x80000000u;

__device__ __forceinline__ uint32_t shared_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive(const uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(shared_at(bar)) : "memory");
}
// Before the first step; every thread of the cluster calls it.
__device__ __forceinline__ void maps_init(Maps& s, int warps, int cluster) {
  if (threadIdx.x == 0) {
    auto init = [](const uint64_t* bar, int count) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_at(bar)), "r"(count)
                   : "memory");
    };
    for (int i = 0; i < 2; ++i) {
      init(&s.given[i], warps);
      init(&s.full[i], 1);
      init(&s.ready[i], 1);
    }
    s.given_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (cluster > 1) cluster_sync();
  else __syncthreads();
}
// 16 bytes into block `rank`'s copy of a variable, counted on its barrier.
__device__ __forceinline__ void send(const void* to, const uint64_t* bar, uint32_t rank, float4 v) {
  uint32_t at, b;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(shared_at(to)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(shared_at(bar)), "r"(rank));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
      "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)),
      "r"(__float_as_uint(v.w)), "r"(b)
      : "memory");
}
__device__ __forceinline__ bool completed(const uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(shared_at(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits for a phase of a barrier, for at most limit_ns of wall time behind the first 256 tests (a peer's
// bytes come within microseconds, and a test that fails takes some, so the time is read at every
// 256th only).  false: it ran out, here or in another warp of the block; the status word says so, and the
// call's results are undefined.
__device__ __forceinline__ bool await(Maps& s, const uint64_t* bar, uint32_t parity,
                                      unsigned* status, uint64_t limit_ns) {
  uint64_t since = 0;
  for (uint32_t i = 0; !completed(bar, parity); ++i) {
    if ((i & 255) == 255) {
      uint64_t now;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
      if (since == 0) since = now;
      if (*reinterpret_cast<volatile int*>(&s.given_up)) return false;
      if (now - since > limit_ns) {
        *reinterpret_cast<volatile int*>(&s.given_up) = 1;
        atomicOr(status, kDevTimeout);
        return false;
      }
    }
  }
  return true;
}

// A computing warp's map of step `step`.
__device__ __forceinline__ void give(Maps& s, int step, int w, int lane, float4 mine) {
  s.warp[step & 1][w][lane] = mine;
  __syncwarp();
  if (lane == 0) arrive(&s.given[step & 1]);
}
// The state in front of its run of that step.  It comes from the exchange warp, whose waits have the limit in
// time: this one ends when that warp has given up, with whatever lies there (or itself gives up after
// 2^28 tests, twenty minutes).
__device__ __forceinline__ f32x2 take(Maps& s, int step, int w, int lane, unsigned* status) {
  for (uint32_t i = 0; !completed(&s.ready[step & 1], (step >> 1) & 1); ++i) {
    if ((i & 255) == 0 && *reinterpret_cast<volatile int*>(&s.given_up)) break;
    if (i == 1u << 28) {
      *reinterpret_cast<volatile int*>(&s.given_up) = 1;
      atomicOr(status, kDevTimeout);
      break;
    }
  }
  return s.front[step & 1][w][lane];
}

// How far a lane of the exchange came: steps whose bytes are expected (lane 0) and that it has sent.
struct Came {
  int armed = 0, sent = 0;
  bool ok = true;
};
__device__ __forceinline__ void expect(Maps& s, int turn, int cluster) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_at(&s.full[turn])),
               "r"(cluster * 512)
               : "memory");
}
// The states in front of the warps' runs of a step, and behind the last: in batches, in which the loads of one
// map do not wait for the stores of another's.
constexpr int kBatch = 5;
template <bool STARTS>
__device__ __forceinline__ f32x2 fronts(Maps& s, int turn, int warps, int lane, f32x2 front) {
  for (int k = 0; k < warps; k += kBatch) {
    float4 m[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) m[i] = s.warp[turn][k + i < warps ? k + i : k][lane];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (k + i < warps) {
        s.front[turn][k + i][lane] = front;
        front = apply<STARTS>(m[i], front);
      }
    }
  }
  __syncwarp();
  if (lane == 0) arrive(&s.ready[turn]);
  return front;
}

// The exchange warp of a block: `steps` exchanges from the state in front of the first one; returns
// the one behind the last.  Of a block alone (whether a wait ran out is looked at now and then only):
template <bool STARTS>
__device__ __forceinline__ f32x2 exchange_alone(Maps& s, long long steps, int warps, int lane,
                                                f32x2 state, const RecurArgs& a) {
  for (long long step = 0; step < steps; ++step) {
    const int turn = (int)step & 1;
    (void)await(s, &s.given[turn], (uint32_t)(step >> 1) & 1, a.status, a.wait_ns);
    state = fronts<STARTS>(s, turn, warps, lane, state);
    if ((step & 63) == 63 && __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s.given_up))) break;
  }
  return state;
}

// Of block `rank` of `cluster`.  Every block sends its map to all blocks of the cluster, where the bytes' arrival
// completes a barrier: no cluster barrier and no fence.  Buffers are written again
// safely: a warp gives step k + 2 after it took step k; a front of step k + 2
// is written after all gave k + 2; and a block sends step k + 2 after it has received all of
// k + 1, which every block sends after it has read all of step k.
// Where a wait ran out a lane waits and sends no more.
template <bool STARTS>
__device__ __forceinline__ f32x2 exchange(Maps& s, long long steps, int warps, int rank, int cluster,
                                          int lane, f32x2 state, const RecurArgs& a, Came& came) {
  for (long long step = 0; step < steps; ++step) {
    const int turn = (int)step & 1;
    const uint32_t parity = (uint32_t)(step >> 1) & 1;
    if (came.ok) {
      if (lane == 0) expect(s, turn, cluster);
      came.armed = (int)step + 1;
      came.ok = await(s, &s.given[turn], parity, a.status, a.wait_ns);
    }
    float4 all = make_float4(1.f, 1.f, 0.f, 0.f);
    for (int k = 0; k < warps; k += kBatch) {
      float4 m[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) m[i] = s.warp[turn][k + i < warps ? k + i : k][lane];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (k + i < warps) all = compose<STARTS>(all, m[i]);
    }
    if (came.ok) {
      for (int k = 0; k < cluster; ++k)
        send(&s.block[turn][rank][lane], &s.full[turn], (rank + k) % cluster, all);
      came.sent = (int)step + 1;
      came.ok = await(s, &s.full[turn], parity, a.status, a.wait_ns);
    }
    f32x2 front = state;
    for (int k = 0; k < cluster; ++k) {
      if (k == rank) front = state;
      state = apply<STARTS>(s.block[turn][k][lane], state);
    }
    (void)fronts<STARTS>(s, turn, warps, lane, front);
  }
  return state;
}

// The blocks of a cluster end together, none while another's maps may be on their way to it: all have
// received those of every step, unless a wait ran out somewhere.  They tell each other how far they came.
// A lane is one step ahead of any other at most (it sends a step when it has received all of the one
// before), so those behind send theirs of that step too, whatever it holds, and all wait for the last bytes.
__device__ __forceinline__ void part(Maps& s, bool exchanges, int lane, int rank, int cluster,
                                     const Came& came) {
  if (exchanges) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, (unsigned)came.sent);
    const uint32_t told = most | (__all_sync(0xffffffffu, came.ok) ? 0u : kGaveUp);
    if (lane < cluster) {
      uint32_t at;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(shared_at(&s.told[rank])), "r"(lane));
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(told) : "memory");
    }
  }
  cluster_sync();
  const volatile uint32_t* told = s.told;
  uint32_t early = 0, most = 0;
  for (int k = 0; k < cluster; ++k) {
    early |= told[k] & kGaveUp;
    most = max(most, told[k] & ~kGaveUp);
  }
  if (!early) return;  // (the same in all blocks)
  if (exchanges) {
    if ((uint32_t)came.sent < most) {
      const int turn = came.sent & 1;
      if (lane == 0 && came.armed == came.sent) expect(s, turn, cluster);
      for (int k = 0; k < cluster; ++k)
        send(&s.block[turn][rank][lane], &s.full[turn], k, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    for (uint32_t step = most < 2 ? 0 : most - 2; step < most; ++step)
      for (int i = 0; i < 4096; ++i)
        if (completed(&s.full[step & 1], step >> 1 & 1)) break;
  }
  cluster_sync();
}

// ---------------------------------------------------------------- the split
struct Split {
  int cols;        // blocks of kChans channels
  int cluster;     // blocks along the tokens
  int warps;       // runs a block
  int spg;         // sequences a group (dense), or 0: all rows are one group (packed)
  long long groups;
  long long rows;  // rows of a group (the last one of a dense batch may have fewer)
};

// Rows [lo, hi) of group g.
__device__ __forceinline__ void group_rows(const Split& p, int B, int T, long long g,
                                           long long* lo, long long* hi) {
  if (p.spg == 0) {
    *lo = 0;
    *hi = T;
    return;
  }
  const long long s = g * p.spg, e = s + p.spg < B ? s + p.spg : B;
  *lo = s * T;
  *hi = e * T;
}

// Walks a warp's rows and knows where sequences begin and end (STARTS: groups hold
// several).  Ascending rows between calls of seek are cheap.
struct Seqs {
  const int32_t* cu;
  int B, T;
  int s = -1;
  long long lo = 0, hi = 0;
  __device__ Seqs(const int32_t* c, int b, int t) : cu(c), B(b), T(t) {}
  // The sequence of row r.  For malformed offsets any index in [0, B).
  __device__ __forceinline__ void seek(long long r) {
    if (s >= 0 && r >= lo && r < hi) return;
    s = seq_of_row(cu, B, T, r);
    seq_rows(cu, s, T, &lo, &hi);
  }
};

constexpr int kKeep = 4;  // tokens between two states kept for the backward pass
constexpr int kBwdWarps = 15, kBwdBlocks = 1;  // that compute in the backward kernel's blocks

// How a call of these sizes is split; `run`: tokens of a run, `most`: warps of a block,
// `blocks`: blocks an SM holds.
Split split(int B, int T, int D, bool packed, int run, int most, int blocks);

// The launchers, by the rows' type: prompts; the state in front of every kKeep rows of
// every group, kept [groups][kept_rows][D]; gradients.
cudaError_t fwd_bf16(const RecurArgs& a, cudaStream_t stream);
cudaError_t fwd_f32(const RecurArgs& a, cudaStream_t stream);
cudaError_t keep_bf16(const RecurArgs& a, float* kept, long long kept_rows, cudaStream_t stream);
cudaError_t keep_f32(const RecurArgs& a, float* kept, long long kept_rows, cudaStream_t stream);
cudaError_t bwd_bf16(const RecurBwdArgs& b, const Split& p, const float* kept,
                     long long kept_rows, float* partial, cudaStream_t stream);
cudaError_t bwd_f32(const RecurBwdArgs& b, const Split& p, const float* kept,
                    long long kept_rows, float* partial, cudaStream_t stream);

}  // namespace recur
}  // namespace gla
