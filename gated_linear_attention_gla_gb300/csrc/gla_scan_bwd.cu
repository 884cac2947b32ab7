// gla_scan_bwd.cu -- the gradients of the selective scan.
//
// With g_t = dy_t silu(z_t) (or dy_t), decay_t = exp(delta_t a) and e_t =
// dL/dh_t = c_t g_t + decay_{t+1} e_{t+1} (e behind the last token: the final
// state's gradient), per channel d and state n:
//     dc_t[n] = sum_d g_t h_t          db_t[n] = sum_d e_t delta_t u_t
//     w_t     = e_t decay_t h_{t-1}    da      = sum_t w_t delta_t
//     s1_t    = sum_n e_t b_t          s2_t    = sum_n a w_t
//     du_t    = delta_t s1_t + skip g_t
//     ddelta_t = s2_t + u_t s1_t,      ddt_t   = ddelta_t softplus'(dt_t + bias)
//     dskip = sum g u,  ddt_bias = sum ddt,  dz_t = dy_t y_t silu'(z_t),
//     d_init = decay_0 e_0
//
// Nothing of the forward pass is kept: the token axis is cut into chunks of 64
// and four launches run over (chunk, channel tile) blocks:
//   1. per chunk, the state it adds (h from zero), the gradient it passes to
//      the chunk before (e from zero, formed forwards with the running product
//      of the decays) and sum delta, whose exponential is the chunk's decay;
//   2. per (channel, n), both recurrences over the chunks: the state entering
//      and the gradient reaching every chunk;
//   3. per chunk: forwards once, keeping the state every 8 tokens, then
//      backwards in groups of 8 tokens whose states and decays are recomputed
//      into registers.  Sums over n are reduced over a channel's lanes, those
//      over d over the warp's channels, then over the warps in shared memory,
//      then written as one fp32 partial per channel tile;
//   4. the partials' sums (b, c over channel tiles; a, skip, dt_bias over chunks).
// No atomics: the same inputs give the same bits.
//
// Bound: instruction issue on the CUDA cores (three exponentials and ~17
// multiply-adds per state and token), not HBM.  A lane owns four states of two
// adjacent channels, one register pair per state (f32x2 instructions work on
// both channels): the sums over d that every lane takes part in are halved, and
// per-channel factors are pairs as they lie in shared memory.
// 8192 bf16 rows x 2048 channels x 16 states: 455 us (plus launches: sums 101, chunks 25,
// gradients 330, partials 13), where the bytes take 35 us and one exponential a
// state 36 us.  The gradients issue at 57 %, two blocks of 128 threads a SM by registers;
// two states a lane and twice the warps 462 us (a fifth more instructions), chunks of 32
// 490 us or more (the chunk arrays double).
#include "gla_scan.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kCH = 64;    // tokens per chunk
constexpr int kSub = 8;    // tokens per recomputed group
constexpr int kV = 4;      // adjacent channels per load

// Workspace, in floats: h and e [slots][D][NS], sums [slots][D] x 2, partials
// of db and dc [channel tiles][rows][2 NS].
struct Space {
  float *h, *e, *sum, *sum2, *part;
  size_t floats;
};
inline Space space_of(float* base, int B, long long rows, int D, int NS) {
  const size_t slots = (size_t)slots_of(B, rows, kCH);
  const size_t tiles = ((size_t)D * NS + 1023) / 1024;
  Space w;
  size_t at = 0;
  auto take = [&](size_t n) {
    float* q = base ? base + at : nullptr;
    at += (n + 63) / 64 * 64;
    return q;
  };
  w.h = take(slots * D * NS);
  w.e = take(slots * D * NS);
  w.sum = take(slots * D);
  w.sum2 = take(slots * D);
  w.part = take(tiles * (size_t)rows * 2 * NS);
  w.floats = at;
  return w;
}

// The lanes' roles: four states 4 q .. of the channels 2 pair, 2 pair + 1 of the
// block's tile.
template <int NS> struct Roles {
  static constexpr int LPC = NS / 4;          // lanes per channel pair
  static constexpr int PPW = 32 / LPC;        // pairs per warp
  static constexpr int CT = kWarps * PPW * 2; // channels per block: 1024 / NS
  static constexpr int PT = CT / 2;
  static constexpr int VPT = CT / kV, STEP = kThreads / VPT;  // threads per token of a load
  // A lane's bits: the pair's lowest, q's lowest, the pair's others, q's others.
  // Reads by pair are then the same in lanes 2 apart and reads by q in lanes 1
  // apart: either lets 16 bytes a lane take two cycles instead of four.
  static __device__ __forceinline__ int pair_of(int lane) {
    return PPW == 1 ? 0 : (lane & 1) | ((lane >> 1) & (PPW - 2));
  }
  static __device__ __forceinline__ int q_of(int lane) {
    return PPW == 1 ? lane : ((lane >> 1) & 1) | (lane / PPW & ~1);
  }
  // The distance of lanes that differ in bit m of the pair, of q.
  static constexpr int pair_bit(int m) { return m == 1 ? 1 : 2 * m; }
  static constexpr int q_bit(int m) { return PPW == 1 ? m : m == 1 ? 2 : PPW * m; }
};

// A chunk's inputs in shared memory.
template <int NS> struct Staged {
  static constexpr int PT = Roles<NS>::PT;
  float4 d[kCH][PT];            // delta, delta u of a channel pair; later s1, s2
  float2 g[kCH][PT];            // g; later y
  float2 b[kCH][NS], c[kCH][NS];  // each value twice
};

// u, dt, dy and z of four channels of a token, as they lie in memory, and as
// values with delta and x = dt + bias.
template <typename IO> struct RawRow {
  Raw<IO, kV> u, dt, g, z;
};
struct Row {
  float u[kV], dl[kV], g[kV], z[kV], x[kV];
};
template <typename IO>
__device__ __forceinline__ RawRow<IO> load_row(const ScanBwdArgs& a, long long row, int ch, bool on) {
  const ScanArgs& p = a.f;
  RawRow<IO> r;
  r.u = r.dt = r.g = r.z = zero_raw<IO, kV>();
  if (on) {
    r.u = load_raw<IO, kV>((const IO*)p.u + row * p.u_stride + ch);
    r.dt = load_raw<IO, kV>((const IO*)p.dt + row * p.dt_stride + ch);
    r.g = load_raw<IO, kV>((const IO*)a.d_out + row * p.D + ch);
    if (p.z) r.z = load_raw<IO, kV>((const IO*)p.z + row * p.z_stride + ch);
  }
  return r;
}
template <typename IO>
__device__ __forceinline__ void unpack_row(const ScanArgs& p, const RawRow<IO>& raw,
                                           const float (&bias)[kV], Row& r) {
  unpack_as<IO, kV>(raw.u, r.u);
  unpack_as<IO, kV>(raw.dt, r.x);
  unpack_as<IO, kV>(raw.g, r.g);
  unpack_as<IO, kV>(raw.z, r.z);
#pragma unroll
  for (int i = 0; i < kV; ++i) r.dl[i] = r.x[i] = r.x[i] + bias[i];
  if (p.softplus) {
#pragma unroll
    for (int i = 0; i < kV; i += 2)
      unpack2(softplus2<sizeof(IO) == 4>(pack2(r.x[i], r.x[i + 1])), &r.dl[i], &r.dl[i + 1]);
  }
}

__device__ __forceinline__ void load_bias(const ScanArgs& p, int ch, bool on, float (&bias)[kV]) {
#pragma unroll
  for (int i = 0; i < kV; ++i) bias[i] = on && p.dt_bias ? __ldg(p.dt_bias + ch + i) : 0.f;
}

// Zeros stand for rows and channels that are not there: decay 1, no drive.  The
// loads of eight rows a thread (and of its share of b and c) are in flight
// together.
template <typename IO, int NS>
__device__ __forceinline__ void stage(const ScanBwdArgs& a, const Chunk& k, int d0, Staged<NS>& s) {
  using L = Roles<NS>;
  const ScanArgs& p = a.f;
  const int vt = (int)threadIdx.x / L::VPT, vc = ((int)threadIdx.x % L::VPT) * kV;
  const bool von = d0 + vc < p.D;
  constexpr int N = kCH / L::STEP < 8 ? kCH / L::STEP : 8;         // rows at once
  constexpr int BC = kCH * NS / kThreads < 8 ? kCH * NS / kThreads : 8;  // b, c elements at once
  float bias[kV];
  load_bias(p, d0 + vc, von, bias);
#pragma unroll 1
  for (int r = 0; r < kCH; r += N * L::STEP) {
    RawRow<IO> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long row = k.t0 + r + i * L::STEP + vt;
      raw[i] = load_row<IO>(a, row, d0 + vc, row < k.t1 && von);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = r + i * L::STEP + vt;
      const bool in = k.t0 + t < k.t1 && von;
      Row v;
      unpack_row<IO>(p, raw[i], bias, v);
      if (p.z) {
#pragma unroll
        for (int j = 0; j < kV; j += 2) {
          const f32x2 z = pack2(v.z[j], v.z[j + 1]);
          unpack2(mul2(pack2(v.g[j], v.g[j + 1]), mul2(z, sigmoid2(z))), &v.g[j], &v.g[j + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < kV; ++j) v.dl[j] = in ? v.dl[j] : 0.f;
      s.d[t][vc / 2] = make_float4(v.dl[0], v.dl[1], v.dl[0] * v.u[0], v.dl[1] * v.u[1]);
      s.d[t][vc / 2 + 1] = make_float4(v.dl[2], v.dl[3], v.dl[2] * v.u[2], v.dl[3] * v.u[3]);
      *reinterpret_cast<float4*>(&s.g[t][vc / 2]) = make_float4(v.g[0], v.g[1], v.g[2], v.g[3]);
    }
  }
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < kCH * NS; i0 += BC * kThreads) {
    IO rb[BC], rc[BC];
#pragma unroll
    for (int x = 0; x < BC; ++x) {
      const int i = i0 + x * kThreads;
      const long long row = k.t0 + i / NS;
      rb[x] = rc[x] = from_f32<IO>(0.f);
      if (row < k.t1) {
        rb[x] = ((const IO*)p.b)[row * p.b_stride + i % NS];
        rc[x] = ((const IO*)p.c)[row * p.c_stride + i % NS];
      }
    }
#pragma unroll
    for (int x = 0; x < BC; ++x) {
      const int i = i0 + x * kThreads;
      const float b = to_f32(rb[x]), c = to_f32(rc[x]);
      s.b[i / NS][i % NS] = make_float2(b, b);
      s.c[i / NS][i % NS] = make_float2(c, c);
    }
  }
}

// Four states of a channel pair from [channel][NS] (base at the pair's first
// channel and the lane's first state), scaled; and back.  `swap` exchanges the
// first two with the last two (see ChannelSums).
__device__ __forceinline__ void exchange(f32x2 (&v)[4]) {
  const f32x2 x = v[0], y = v[1];
  v[0] = v[2];
  v[1] = v[3];
  v[2] = x;
  v[3] = y;
}
__device__ __forceinline__ void load_states(const float* base, int NS, float scale, bool swap,
                                            f32x2 (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(base);
  const float4 y = *reinterpret_cast<const float4*>(base + NS);
  v[0] = pack2(x.x * scale, y.x * scale);
  v[1] = pack2(x.y * scale, y.y * scale);
  v[2] = pack2(x.z * scale, y.z * scale);
  v[3] = pack2(x.w * scale, y.w * scale);
  if (swap) exchange(v);
}
__device__ __forceinline__ void store_states(float* base, int NS, bool swap, f32x2 (&v)[4]) {
  if (swap) exchange(v);
  *reinterpret_cast<float4*>(base) = make_float4(v[0].x, v[1].x, v[2].x, v[3].x);
  *reinterpret_cast<float4*>(base + NS) = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
}
// The lane's four values of a row of b or c, each twice; lo and hi are the
// places of its first and its last two.
__device__ __forceinline__ void load_dup(const float2* row, int lo, int hi, f32x2 (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(row + lo);
  const float4 y = *reinterpret_cast<const float4*>(row + hi);
  v[0] = pack2(x.x, x.y);
  v[1] = pack2(x.z, x.w);
  v[2] = pack2(y.x, y.y);
  v[3] = pack2(y.z, y.w);
}

// 1. What each chunk adds to the state and to the gradient before it.
template <typename IO, int NS>
__global__ void __launch_bounds__(kThreads, 3) chunk_sums_kernel(ScanBwdArgs a, Space w) {
  using L = Roles<NS>;
  const ScanArgs& p = a.f;
  extern __shared__ __align__(16) unsigned char smem[];
  Staged<NS>& s = *reinterpret_cast<Staged<NS>*>(smem);
  const int tiles = (p.D + L::CT - 1) / L::CT;
  const long long slot = blockIdx.x / tiles;
  const int d0 = (int)(blockIdx.x % tiles) * L::CT;
  const Chunk k = chunk_of_slot(p, slot, kCH);
  if (!k.ok) return;
  const int lane = threadIdx.x & 31, q = L::q_of(lane);
  const int pair = (threadIdx.x >> 5) * L::PPW + L::pair_of(lane), ch = d0 + 2 * pair;
  const bool on = ch < p.D;  // (D is even: both channels or none)
  stage<IO, NS>(a, k, d0, s);
  f32x2 a2[4] = {}, h[4] = {}, e[4] = {}, run[4], sum = {};
#pragma unroll
  for (int j = 0; j < 4; ++j) run[j] = both(1.f);
  if (on) load_states(p.a + (long long)ch * NS + q * 4, NS, kLog2e, false, a2);
  __syncthreads();
#pragma unroll 4
  for (int t = 0; t < kCH; ++t) {
    const float4 d = s.d[t][pair];
    const float2 gg = s.g[t][pair];
    const f32x2 dl = pack2(d.x, d.y), du = pack2(d.z, d.w), g = pack2(gg.x, gg.y);
    f32x2 b[4], c[4];
    load_dup(s.b[t], q * 4, q * 4 + 2, b);
    load_dup(s.c[t], q * 4, q * 4 + 2, c);
    sum = add2(sum, dl);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x2 decay = decay2<sizeof(IO) == 4>(mul2(dl, a2[j]));
      h[j] = fma2(decay, h[j], mul2(du, b[j]));
      run[j] = mul2(run[j], decay);
      e[j] = fma2(mul2(run[j], c[j]), g, e[j]);
    }
  }
  if (on) {
    const long long at = (slot * p.D + ch) * NS + q * 4;
    store_states(w.h + at, NS, false, h);
    store_states(w.e + at, NS, false, e);
    if (q == 0) {
      float2 v;
      unpack2(sum, &v.x, &v.y);
      *reinterpret_cast<float2*>(w.sum + slot * p.D + ch) = v;
    }
  }
}

// 2. The state entering each chunk (blockIdx.y 0) and the gradient reaching its
// last token from behind (blockIdx.y 1), in place; d_init.
__global__ void __launch_bounds__(128)
chunk_scan_kernel(ScanBwdArgs a, Space w, long long slots) {
  after_previous();
  const ScanArgs& p = a.f;
  const int quads = p.NS / 4;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long per = (long long)p.D * quads;
  if (i >= per * p.B) return;
  const int s = (int)(i / per);
  const long long in = i % per;  // channel * quads + quad
  const int ch = (int)(in / quads);
  long long lo, hi;
  if (!seq_ok(p, s, in == 0, &lo, &hi)) return;
  const long long f = first_slot(p, s, kCH);
  const long long n = min((hi - lo + kCH - 1) / kCH, slots - f);
  float4 x = __ldg(reinterpret_cast<const float4*>(p.a) + in);
  x.x *= kLog2e; x.y *= kLog2e; x.z *= kLog2e; x.w *= kLog2e;
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool back = blockIdx.y != 0;
  const float* start = back ? a.d_final_state : p.init_state;
  if (start) run = reinterpret_cast<const float4*>(start)[(long long)s * per + in];
  scan_chunks(reinterpret_cast<float4*>(back ? w.e : w.h), w.sum, x, f, n, per, in, p.D, ch, back,
              &run);
  if (back && a.d_init_state) reinterpret_cast<float4*>(a.d_init_state)[(long long)s * per + in] = run;
}

// The sums over the warp's channels of two tokens' values v[token * 4 + state]
// (of db and dc), scattered: afterwards a lane holds N = 4, 2 or 1 of them.  Lanes
// in the upper half of the pairs hold their states exchanged, the first two
// for the last two, so that in the first step every lane keeps its first two
// states and gives the last two, without selecting which.  Value i of the result
// is token token_of(i)'s, of state state_of(i) of the lane's four.
template <int NS> struct ChannelSums {
  using L = Roles<NS>;
  static constexpr int PPW = L::PPW;
  static constexpr int N = PPW == 2 ? 4 : PPW == 4 ? 2 : 1;
  f32x2 r[4];
  int p;
  __device__ __forceinline__ ChannelSums(const f32x2 (&v)[8], int p) : p(p) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        r[t * 2 + j] = add2(v[t * 4 + j], shfl_xor2(v[t * 4 + j + 2], L::pair_bit(PPW / 2)));
    if constexpr (PPW >= 4) {
      const bool up = (p & (PPW / 4)) != 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x2 give = up ? r[j] : r[j + 2], keep = up ? r[j + 2] : r[j];
        r[j] = add2(keep, shfl_xor2(give, L::pair_bit(PPW / 4)));
      }
    }
    if constexpr (PPW >= 8) {
      const bool up = (p & (PPW / 8)) != 0;
      const f32x2 give = up ? r[0] : r[1], keep = up ? r[1] : r[0];
      r[0] = add2(keep, shfl_xor2(give, L::pair_bit(PPW / 8)));
    }
    if constexpr (PPW == 16) r[0] = add2(r[0], shfl_xor2(r[0], 1));
  }
  __device__ __forceinline__ int token_of(int i) const {
    return PPW == 2 ? i / 2 : (p & (PPW / 4)) != 0;
  }
  __device__ __forceinline__ int state_of(int i) const {
    return (PPW <= 4 ? i % 2 : (p & (PPW / 8)) != 0) + ((p & (PPW / 2)) != 0 ? 2 : 0);
  }
};

// The sums of v[0 .. 4) over a channel pair's lanes (bits PPW and up),
// scattered: a lane holds 4 / LPC of them, or one that lanes share.
template <int NS>
__device__ __forceinline__ void reduce_states(f32x2 (&v)[4], int q, int* first) {
  using L = Roles<NS>;
  constexpr int LPC = L::LPC;
  const bool up = (q & (LPC / 2)) != 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const f32x2 give = up ? v[k] : v[k + 2], keep = up ? v[k + 2] : v[k];
    v[k] = add2(keep, shfl_xor2(give, L::q_bit(LPC / 2)));
  }
  *first = up ? 2 : 0;
  if constexpr (LPC >= 4) {
    const bool up2 = (q & (LPC / 4)) != 0;
    const f32x2 give = up2 ? v[0] : v[1], keep = up2 ? v[1] : v[0];
    v[0] = add2(keep, shfl_xor2(give, L::q_bit(LPC / 4)));
    *first += up2 ? 1 : 0;
#pragma unroll
    for (int off = LPC / 8; off > 0; off >>= 1)
      v[0] = add2(v[0], shfl_xor2(v[0], L::q_bit(off)));
  }
}

template <int NS> struct GradSmem {
  Staged<NS> in;
  float4 h[kCH / kSub][2][kThreads];  // the state in front of every group, by thread
  float red[kWarps][kSub][2 * NS];    // the warps' sums over d
  float tail[2][Roles<NS>::STEP][Roles<NS>::CT];
};

// 3. The chunk's gradients.
template <typename IO, typename OUT, int NS>
__global__ void __launch_bounds__(kThreads, 2) chunk_grads_kernel(ScanBwdArgs a, Space w) {
  after_previous();
  using L = Roles<NS>;
  constexpr int LPC = L::LPC, PPW = L::PPW, CT = L::CT;
  constexpr int kShare = LPC > 4 ? LPC / 4 : 1;  // lanes that share a sum over n
  const ScanArgs& p = a.f;
  extern __shared__ __align__(16) unsigned char smem[];
  GradSmem<NS>& m = *reinterpret_cast<GradSmem<NS>*>(smem);
  Staged<NS>& s = m.in;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = L::q_of(lane);
  const int tiles = (p.D + CT - 1) / CT, tile = (int)(blockIdx.x % tiles);
  const long long slot = blockIdx.x / tiles, rows = rows_of(p);
  const int d0 = tile * CT, p_in = L::pair_of(lane), pair = warp * PPW + p_in, ch = d0 + 2 * pair;
  const bool on = ch < p.D;
  const long long at = (slot * p.D + ch) * NS + q * 4;
  const Chunk k = chunk_of_slot(p, slot, kCH);
  if (!k.ok) {  // no chunk: its partials count as zero
    if (on) {
      f32x2 none[4] = {};
      store_states(w.h + at, NS, false, none);
      if (q == 0) {
        const float2 zero = make_float2(0.f, 0.f);
        *reinterpret_cast<float2*>(w.sum + slot * p.D + ch) = zero;
        *reinterpret_cast<float2*>(w.sum2 + slot * p.D + ch) = zero;
      }
    }
    return;
  }
  const bool swap = (p_in & (PPW / 2)) != 0;
  const int lo4 = q * 4 + (swap ? 2 : 0), hi4 = q * 4 + (swap ? 0 : 2);
  f32x2 a2[4] = {}, h[4] = {}, e[4] = {}, da[4] = {};
  if (on) {
    load_states(p.a + (long long)ch * NS + q * 4, NS, kLog2e, swap, a2);
    load_states(w.h + at, NS, 1.f, swap, h);
    load_states(w.e + at, NS, 1.f, swap, e);
  }
  stage<IO, NS>(a, k, d0, s);
  __syncthreads();
  const int len = (int)(k.t1 - k.t0);
  const int groups = (len + kSub - 1) / kSub;

  // forwards, keeping the state in front of every group
  for (int gr = 0; gr < groups; ++gr) {
    float4 x, y;
    unpack2(h[0], &x.x, &x.y);
    unpack2(h[1], &x.z, &x.w);
    unpack2(h[2], &y.x, &y.y);
    unpack2(h[3], &y.z, &y.w);
    m.h[gr][0][tid] = x;
    m.h[gr][1][tid] = y;
    if (gr + 1 == groups) break;
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      const int t = gr * kSub + i;
      const float4 d = s.d[t][pair];
      const f32x2 dl = pack2(d.x, d.y), du = pack2(d.z, d.w);
      f32x2 b[4];
      load_dup(s.b[t], lo4, hi4, b);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[j] = fma2(decay2<sizeof(IO) == 4>(mul2(dl, a2[j])), h[j], mul2(du, b[j]));
    }
  }
  // backwards
#pragma unroll 1
  for (int gr = groups - 1; gr >= 0; --gr) {
    f32x2 hs[kSub + 1][4], ds[kSub][4];
    {
      const float4 x = m.h[gr][0][tid], y = m.h[gr][1][tid];
      hs[0][0] = pack2(x.x, x.y);
      hs[0][1] = pack2(x.z, x.w);
      hs[0][2] = pack2(y.x, y.y);
      hs[0][3] = pack2(y.z, y.w);
    }
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      const int t = gr * kSub + i;
      const float4 d = s.d[t][pair];
      const f32x2 dl = pack2(d.x, d.y), du = pack2(d.z, d.w);
      f32x2 b[4];
      load_dup(s.b[t], lo4, hi4, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ds[i][j] = decay2<sizeof(IO) == 4>(mul2(dl, a2[j]));
        hs[i + 1][j] = fma2(ds[i][j], hs[i][j], mul2(du, b[j]));
      }
    }
#pragma unroll
    for (int half = kSub / 4 - 1; half >= 0; --half) {
      f32x2 s1[4], s2[4], y[4];
      f32x2 v[8];  // a token's and state's terms of db and dc
#pragma unroll
      for (int x = 3; x >= 0; --x) {
        const int i = half * 4 + x, t = gr * kSub + i;
        const float4 d = s.d[t][pair];
        const float2 gg = s.g[t][pair];
        const f32x2 dl = pack2(d.x, d.y), du = pack2(d.z, d.w), g = pack2(gg.x, gg.y);
        f32x2 b[4], c[4];
        load_dup(s.b[t], lo4, hi4, b);
        load_dup(s.c[t], lo4, hi4, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[j] = fma2(c[j], g, e[j]);
          const f32x2 tb = mul2(du, e[j]), tc = mul2(g, hs[i + 1][j]);
          v[(x & 1) * 4 + j] = make_float2(tb.x + tb.y, tc.x + tc.y);
          s1[x] = j == 0 ? mul2(e[0], b[0]) : fma2(e[j], b[j], s1[x]);
          y[x] = j == 0 ? mul2(c[0], hs[i + 1][0]) : fma2(c[j], hs[i + 1][j], y[x]);
          e[j] = mul2(e[j], ds[i][j]);
          const f32x2 wj = mul2(e[j], hs[i][j]);
          da[j] = fma2(dl, wj, da[j]);
          s2[x] = j == 0 ? mul2(a2[0], wj) : fma2(a2[j], wj, s2[x]);
        }
        if ((x & 1) == 0) {  // tokens i and i + 1
          const ChannelSums<NS> sums(v, p_in);
          if (PPW <= 8 || (p_in & 1) == 0) {
#pragma unroll
            for (int n = 0; n < ChannelSums<NS>::N; ++n) {
              float* to = m.red[warp][i + sums.token_of(n)] + q * 4 + sums.state_of(n);
              to[0] = sums.r[n].x;
              to[NS] = sums.r[n].y;
            }
          }
        }
      }
      int first;
      reduce_states<NS>(s1, q, &first);
      reduce_states<NS>(s2, q, &first);
      reduce_states<NS>(y, q, &first);
      __syncwarp();  // the pair's lanes have read these tokens' d and g
      if (q % kShare == 0) {
#pragma unroll
        for (int v = 0; v < (LPC == 2 ? 2 : 1); ++v) {
          const int t = gr * kSub + half * 4 + first + v;
          float4 o;
          unpack2(s1[v], &o.x, &o.y);
          unpack2(s2[v], &o.z, &o.w);
          s.d[t][pair] = o;
          float2 yy;
          unpack2(y[v], &yy.x, &yy.y);
          s.g[t][pair] = yy;
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < kSub * 2 * NS; i += kThreads) {
      const int t = i / (2 * NS), col = i % (2 * NS);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) sum += m.red[v][t][col];
      const long long row = k.t0 + gr * kSub + t;
      if (row < k.t1) w.part[((long long)tile * rows + row) * 2 * NS + col] = sum;
    }
    __syncthreads();
  }
  if (on) store_states(w.h + at, NS, swap, da);  // over the state that has been read

  // du, ddt, dz: the inputs once more (from L2), rows of adjacent channels
  const int vt = tid / L::VPT, vc = (tid % L::VPT) * kV;
  const bool von = d0 + vc < p.D;
  float bias[kV], skip[kV], dskip[kV] = {}, dbias[kV] = {};
  load_bias(p, d0 + vc, von, bias);
#pragma unroll
  for (int i = 0; i < kV; ++i) skip[i] = von && p.skip ? __ldg(p.skip + d0 + vc + i) : 0.f;
  constexpr int N = kCH / L::STEP < 8 ? kCH / L::STEP : 8;
#pragma unroll 1
  for (int r = vt; r < len && von; r += N * L::STEP) {
    RawRow<IO> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      raw[i] = load_row<IO>(a, k.t0 + r + i * L::STEP, d0 + vc, r + i * L::STEP < len);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int t = r + n * L::STEP;
      if (t >= len) break;
      Row v;
      unpack_row<IO>(p, raw[n], bias, v);
      const float4 o0 = s.d[t][vc / 2], o1 = s.d[t][vc / 2 + 1];
      const float4 yy = *reinterpret_cast<const float4*>(&s.g[t][vc / 2]);
      const float s1[kV] = {o0.x, o0.y, o1.x, o1.y}, s2[kV] = {o0.z, o0.w, o1.z, o1.w};
      const float y[kV] = {yy.x, yy.y, yy.z, yy.w};
      float du[kV], ddt[kV], dz[kV], slope[kV];
      if (p.softplus) {
#pragma unroll
        for (int i = 0; i < kV; i += 2)
          unpack2(softplus_slope2<sizeof(IO) == 4>(pack2(v.x[i], v.x[i + 1])), &slope[i],
                  &slope[i + 1]);
      }
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        float g = v.g[i];
        if (p.z) {
          const float sg = sigmoid(v.z[i]);
          dz[i] = g * sg * fmaf(v.z[i], 1.f - sg, 1.f) * fmaf(skip[i], v.u[i], y[i]);
          g *= v.z[i] * sg;
        }
        ddt[i] = fmaf(kLn2, s2[i], v.u[i] * s1[i]);
        if (p.softplus) ddt[i] *= slope[i];
        du[i] = fmaf(v.dl[i], s1[i], skip[i] * g);
        dskip[i] = fmaf(g, v.u[i], dskip[i]);
        dbias[i] += ddt[i];
      }
      const long long o = (k.t0 + t) * p.D + d0 + vc;
      store_raw<OUT, kV>((OUT*)a.du + o, pack_as<OUT, kV>(du));
      store_raw<OUT, kV>((OUT*)a.ddt + o, pack_as<OUT, kV>(ddt));
      if (a.dz) store_raw<OUT, kV>((OUT*)a.dz + o, pack_as<OUT, kV>(dz));
    }
  }
  // this chunk's share of dskip and ddt_bias
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    m.tail[0][vt][vc + i] = dskip[i];
    m.tail[1][vt][vc + i] = dbias[i];
  }
  __syncthreads();
  for (int i = tid; i < 2 * CT; i += kThreads) {
    const int which = i / CT, c = i % CT;
    float sum = 0.f;
#pragma unroll 8
    for (int t = 0; t < L::STEP; ++t) sum += m.tail[which][t][c];
    if (d0 + c < p.D) (which ? w.sum2 : w.sum)[slot * p.D + d0 + c] = sum;
  }
}

// 4. The partials' sums.  The first blocks: db and dc over the channel tiles, a
// value a thread; the others: da, dskip and ddt_bias over the chunks, 32 columns
// a block, eight threads a column.
template <typename OUT>
__global__ void __launch_bounds__(256)
sum_partials_kernel(ScanBwdArgs a, Space w, int tiles, long long rows, long long slots,
                    long long row_blocks) {
  after_previous();
  const int NS = a.f.NS;
  if ((long long)blockIdx.x < row_blocks) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long n = rows * 2 * NS;
    if (i >= n) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    int t = 0;
    for (; t + 4 <= tiles; t += 4)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += w.part[(t + u) * n + i];
    for (; t < tiles; ++t) s[0] += w.part[t * n + i];
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    const long long row = i / (2 * NS);
    const int col = (int)(i % (2 * NS));
    if (col < NS) ((OUT*)a.db)[row * NS + col] = from_f32<OUT>(sum);
    else ((OUT*)a.dc)[row * NS + col - NS] = from_f32<OUT>(sum);
    return;
  }
  __shared__ float part[8][32];
  const long long D = a.f.D, DN = D * a.f.NS;
  const int col = threadIdx.x % 32, row = threadIdx.x / 32;
  const long long i = ((long long)blockIdx.x - row_blocks) * 32 + col;
  const float* from = nullptr;
  float* to = nullptr;
  long long step = D;
  if (i < DN) { from = w.h + i; to = a.da + i; step = DN; }
  else if (i < DN + D) { from = w.sum + i - DN; to = a.dskip ? a.dskip + i - DN : nullptr; }
  else if (i < DN + 2 * D) {
    from = w.sum2 + i - DN - D;
    to = a.ddt_bias ? a.ddt_bias + i - DN - D : nullptr;
  }
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (to) {
    long long t = row;
    for (; t + 24 < slots; t += 32)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += from[(t + 8 * u) * step];
    for (; t < slots; t += 8) s[0] += from[t * step];
  }
  part[row][col] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (row == 0 && to) {
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) sum += part[r][col];
    *to = sum;
  }
}

template <typename IO, typename OUT, int NS>
cudaError_t launch_typed(const ScanBwdArgs& a, void* workspace, cudaStream_t stream) {
  constexpr int CT = Roles<NS>::CT;
  const ScanArgs& p = a.f;
  const long long rows = p.cu_seqlens ? (long long)p.T : (long long)p.B * p.T;
  const long long slots = slots_of(p.B, rows, kCH);
  const int tiles = (p.D + CT - 1) / CT;
  const Space w = space_of(static_cast<float*>(workspace), p.B, rows, p.D, NS);
  constexpr int smem1 = (int)sizeof(Staged<NS>), smem3 = (int)sizeof(GradSmem<NS>);
  static_assert(smem3 <= 227 * 1024, "shared memory of a block");
  static std::atomic<uint64_t> done1{0}, done3{0};
  cudaError_t e = allow_shared(chunk_sums_kernel<IO, NS>, smem1, done1);
  if (e == cudaSuccess) e = allow_shared(chunk_grads_kernel<IO, OUT, NS>, smem3, done3);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(slots * tiles);
  if (rows > 0) chunk_sums_kernel<IO, NS><<<grid, kThreads, smem1, stream>>>(a, w);
  const long long per = (long long)p.B * p.D * (NS / 4);
  e = cudaGetLastError();
  if (p.B > 0 && e == cudaSuccess)
    e = launch_after(chunk_scan_kernel, dim3((unsigned)((per + 127) / 128), 2), dim3(128), 0,
                     stream, a, w, slots);
  if (p.B > 0 && e == cudaSuccess)
    e = launch_after(chunk_grads_kernel<IO, OUT, NS>, dim3(grid), dim3(kThreads), smem3, stream, a,
                     w);
  if (e != cudaSuccess) return e;
  const long long row_blocks = (rows * 2 * NS + 255) / 256;
  const long long col_blocks = ((long long)p.D * (NS + 2) + 31) / 32;
  return launch_after(sum_partials_kernel<OUT>, dim3((unsigned)(row_blocks + col_blocks)),
                      dim3(256), 0, stream, a, w, tiles, rows, slots, row_blocks);
}

template <typename IO, typename OUT>
cudaError_t launch_io(const ScanBwdArgs& a, void* workspace, cudaStream_t stream) {
  switch (a.f.NS) {
    case 8: return launch_typed<IO, OUT, 8>(a, workspace, stream);
    case 16: return launch_typed<IO, OUT, 16>(a, workspace, stream);
    case 32: return launch_typed<IO, OUT, 32>(a, workspace, stream);
    default: return launch_typed<IO, OUT, 64>(a, workspace, stream);
  }
}

}  // namespace

size_t scan_bwd_workspace(int B, long long rows, int D, int NS) {
  return space_of(nullptr, B, rows, D, NS).floats * 4;
}

cudaError_t launch_scan_bwd(const ScanBwdArgs& a, void* workspace, cudaStream_t stream) {
  if (a.f.fp32_io) return launch_io<float, float>(a, workspace, stream);
  if (a.f.fp32_out) return launch_io<__nv_bfloat16, float>(a, workspace, stream);
  return launch_io<__nv_bfloat16, __nv_bfloat16>(a, workspace, stream);
}

}  // namespace gla
