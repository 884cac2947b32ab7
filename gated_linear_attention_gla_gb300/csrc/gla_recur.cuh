// gla_recur.cuh -- what the kernels of the gated linear recurrence share: the gates of a
// token, the tiles of rows, and how the token axis is split.
//
// A recurrence h_t = a_t h_{t-1} + b_t over a run of tokens is the map
// h -> P h + H of its own (P the product of the a_t), and such maps compose. So
// the token axis is split three ways: a warp takes a run of consecutive tokens
// (its lanes two channels each), a block of `warps` warps consecutive runs, and
// the blocks of a thread-block cluster consecutive blocks of runs.  Each step of
// the loop covers cluster x warps runs: the warps reduce their runs to maps, the
// block composes its warps' (shared memory), the cluster's blocks exchange theirs
// (distributed shared memory, one cluster barrier), every thread folds what lies in front of
// its run onto the state at the step's start, and finishes its tokens from
// registers.  Every input is read once.
#pragma once

#include "gla_ssm.cuh"

namespace gla {
namespace recur {

constexpr int kChans = 64;     // channels of a block: two a lane
constexpr int kMaxWarps = 16;  // runs of a block
constexpr int kMaxCluster = 8;

// ---------------------------------------------------------------- the gates
// A token's values for a pair of channels.
struct Gate {
  f32x2 sf, nf;  // sigmoid(f), 1 - sigmoid(f)
  f32x2 si, ni;  // sigmoid(i), 1 - sigmoid(i)  (1, 0 without i)
  f32x2 l;       // log2 of the decay (with `decay` only)
  f32x2 a, m;    // decay, factor of the drive
  f32x2 k;       // -dm / d(log a)
};

// e / (1 + e) and 1 / (1 + e), whichever is which for the sign of v
__device__ __forceinline__ f32x2 pick(f32x2 v, f32x2 x, f32x2 y) {
  return make_float2(v.x < 0.f ? y.x : x.x, v.y < 0.f ? y.y : x.y);
}

// Sigmoids of a pair (or of two pairs) from e = exp(-|v|) <= 1: the denominators
// lie in [1, 2], so one reciprocal of their product serves all of them (the special-function unit
// is as busy as HBM here: it does a quarter of an instruction's lanes a clock).
template <bool EXACT>
__device__ __forceinline__ void sigmoids2(f32x2 v, f32x2* s, f32x2* n) {
  const f32x2 e = exp_neg_abs2<EXACT>(v), d = add2(e, both(1.f));
  const float r = rcp(d.x * d.y);
  const f32x2 q = make_float2(r * d.y, r * d.x), p = mul2(e, q);
  *s = pick(v, q, p);
  *n = pick(v, p, q);
}
template <bool EXACT>
__device__ __forceinline__ void sigmoids4(f32x2 v, f32x2 w, f32x2* s, f32x2* n, f32x2* t,
                                          f32x2* o) {
  const f32x2 e = exp_neg_abs2<EXACT>(v), g = exp_neg_abs2<EXACT>(w);
  const f32x2 d = add2(e, both(1.f)), c = add2(g, both(1.f)), dc = mul2(d, c);
  const float r = rcp(dc.x * dc.y);
  const f32x2 rr = make_float2(r * dc.y, r * dc.x);  // 1 / dc
  const f32x2 q = mul2(rr, c), u = mul2(rr, d), p = mul2(e, q), x = mul2(g, u);
  *s = pick(v, q, p);
  *n = pick(v, p, q);
  *t = pick(w, u, x);
  *o = pick(w, x, u);
}

// 2^l - 1 and 2^l of l in [-126, 0] without the special-function unit and without
// cancellation near l = 0: l = k + r with |r| <= 1/2, 2^r - 1 by its Taylor
// polynomial (degree 7: off by 5e-9), 2^k in the exponent.  1 - a^2 = -(a - 1)(2 + (a - 1))
// then keeps its relative accuracy for decays of 0.9999.
__device__ __forceinline__ void exp2m1(f32x2 l, f32x2* a, f32x2* u) {
  const f32x2 t = add2(l, both(12582912.f));  // its low bits: k
  const f32x2 r = fma2(add2(t, both(-12582912.f)), both(-1.f), l);
  f32x2 p = fma2(both(1.5252734e-5f), r, both(1.5403530e-4f));
  p = fma2(p, r, both(1.3333558e-3f));
  p = fma2(p, r, both(9.6181291e-3f));
  p = fma2(p, r, both(5.5504109e-2f));
  p = fma2(p, r, both(0.24022651f));
  p = fma2(p, r, both(kLn2));
  p = mul2(p, r);
  const f32x2 s = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                              __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));
  *a = fma2(s, p, s);
  *u = fma2(s, p, add2(s, both(-1.f)));
}

__device__ __forceinline__ float rsqrt_or_0(float v) {  // 0 where v is 0
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return v < 1e-37f ? 0.f : r;
}

// `c`: decay log2(e) of the pair (DECAY)
template <bool EXACT, bool DECAY, bool BWD>
__device__ __forceinline__ Gate gates(f32x2 f, f32x2 i, f32x2 c, bool has_i, bool unit) {
  Gate g;
  if (has_i) {
    sigmoids4<EXACT>(f, i, &g.sf, &g.nf, &g.si, &g.ni);
  } else {
    sigmoids2<EXACT>(f, &g.sf, &g.nf);
    g.si = both(1.f);
    g.ni = both(0.f);
  }
  f32x2 u;  // a - 1
  if (DECAY) {
    g.l = mul2(c, g.sf);
    g.l = make_float2(g.l.x < -126.f ? -126.f : g.l.x, g.l.y < -126.f ? -126.f : g.l.y);
    exp2m1(g.l, &g.a, &u);
  } else {
    g.a = g.sf;
    u = mul2(g.nf, both(-1.f));
  }
  if (unit) {
    const f32x2 v = mul2(mul2(u, both(-1.f)), add2(u, both(2.f)));
    const f32x2 rs = make_float2(rsqrt_or_0(v.x), rsqrt_or_0(v.y));
    g.m = mul2(v, rs);
    if (BWD) g.k = mul2(mul2(g.a, g.a), rs);
  } else {
    g.m = mul2(u, both(-1.f));
    if (BWD) g.k = g.a;
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

// Asynchronous copy of n <= L rows of a block's channels, by one warp.
template <typename T, int L>
__device__ __forceinline__ void copy_rows(T* dst, const void* src, long long stride,
                                          long long row, int n, int c0, int D, int lane) {
  constexpr int E = 16 / (int)sizeof(T), PER = kChans / E, ROWS = 32 / PER;
  const int at = lane % PER * E;
#pragma unroll
  for (int k = 0; k < L; k += ROWS) {
    const int t = k + lane / PER;
    if (t < n && c0 + at < D)
      cp_async16(dst + t * kChans + at, (const T*)src + (row + t) * stride + c0 + at);
  }
}

template <typename OT>
__device__ __forceinline__ void store_pair(OT* p, f32x2 v) {
  const float x[2] = {v.x, v.y};
  store_raw<OT, 2>(p, pack_as<OT, 2>(x));
}

// ---------------------------------------------------------------- composition
// A run's map of a lane's two channels; P < 0: it starts anew (a sequence begins inside),
// so that nothing in front of it is multiplied, infinities included.
__device__ __forceinline__ f32x2 apply(float4 map, f32x2 h) {
  return make_float2(map.x < 0.f ? map.z : fmaf(map.x, h.x, map.z),
                     map.y < 0.f ? map.w : fmaf(map.y, h.y, map.w));
}
// `next` after `map`
__device__ __forceinline__ float4 compose(float4 map, float4 next) {
  float4 r;
  r.x = next.x < 0.f || map.x < 0.f ? -1.f : map.x * next.x;
  r.y = next.y < 0.f || map.y < 0.f ? -1.f : map.y * next.y;
  r.z = next.x < 0.f ? next.z : fmaf(next.x, map.z, next.z);
  r.w = next.y < 0.f ? next.w : fmaf(next.y, map.w, next.w);
  return r;
}

__device__ __forceinline__ void store_remote(const void* local, uint32_t rank, float4 v) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(at)
      : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(local))), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The maps of one step: of the block's warps and of the cluster's blocks, two
// buffers in turn (a block writes one again only after the barrier behind the
// step in which everyone has read it).
struct Maps {
  float4 warp[2][kMaxWarps][32];
  float4 block[2][kMaxCluster][32];
};

// One exchange: `mine` is the warp's map (warp `w` of `warps`, block `rank` of
// `cluster`); returns the state in front of the warp's run and moves *state, the one in front of the
// step, behind it.  Every thread of the cluster calls it.
__device__ __forceinline__ f32x2 exchange(Maps& s, int turn, float4 mine, int w, int warps,
                                          int rank, int cluster, int lane, f32x2* state) {
  s.warp[turn][w][lane] = mine;
  __syncthreads();
  f32x2 h = *state;
  if (cluster == 1) {
    f32x2 front = h;
    for (int k = 0; k < warps; ++k) {
      if (k == w) front = h;
      h = apply(s.warp[turn][k][lane], h);
    }
    *state = h;
    return front;
  }
  if (w == 0) {
    float4 all = s.warp[turn][0][lane];
    for (int k = 1; k < warps; ++k) all = compose(all, s.warp[turn][k][lane]);
    for (int k = 0; k < cluster; ++k) store_remote(&s.block[turn][rank][lane], k, all);
  }
  cluster_sync();
  f32x2 front = h;
  for (int k = 0; k < cluster; ++k) {
    if (k == rank) front = h;
    h = apply(s.block[turn][k][lane], h);
  }
  for (int k = 0; k < w; ++k) front = apply(s.warp[turn][k][lane], front);
  *state = h;
  return front;
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

// How a call of these sizes is split; `run`: tokens of a run, `most`: warps of a block.
Split split(int B, int T, int D, bool packed, int run, int most);
// The state in front of every kKeep rows of every group: kept [groups][kept_rows][D].
cudaError_t launch_keep(const RecurArgs& a, const Split& p, float* kept, long long kept_rows,
                        cudaStream_t stream);

}  // namespace recur
}  // namespace gla
