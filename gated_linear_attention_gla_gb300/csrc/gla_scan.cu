// gla_scan.cu -- the selective scan over prompts (dense or packed).
//
//     delta = softplus(dt + dt_bias)
//     h_t[d][n] = exp(delta_t[d] a[d][n]) h_{t-1}[d][n] + delta_t[d] u_t[d] b_t[n]
//     y_t[d] = (sum_n c_t[n] h_t[d][n] + skip[d] u_t[d]) * silu(z_t[d])
//
// Every (channel, n) has a decay of its own at every token, so no product of
// matrices forms the in-chunk part (as it does in chunk_fwd): the work is NS
// exponentials and 4 NS multiplies and adds per token and channel, on the CUDA
// cores; instruction issue and the exponential unit bound it, not HBM.
//
// A block owns 1024 / NS channels of one run of tokens.  Four compute warps: NS / 8
// lanes a channel, eight states each in four register pairs (f32x2 instructions
// work on two states); the next two tokens are in registers before the current
// ones are used.  Two or three helper groups of four warps take turns: one turns
// (dt, u) of a tile of 1024 (token, channel) pairs into (delta, delta u) in shared
// memory, and finishes and stores the outputs of its tile before, so that the
// recurrence does not wait for loads, the softplus or the gate; named barriers
// hand the stages over.  The sums over n go through shared memory, up to two terms
// per pair, and the helpers add them.
//
// 8192 bf16 rows (four sequences) x 2048 channels x 16 states: 103 us, where the
// tensors' bytes at copy bandwidth are 20 us and the exponentials 36 us of the
// exponential unit.  What bounds it now: 128 blocks of 64 channels, one a SM, each with
// one compute warp a scheduler, whose ~50 instructions a token issue at 55 % together
// with the helpers'.  A warp that owns channel pairs instead of state pairs 132 us
// (against 122 then), step sizes stored twice 130 us, tiles fetched across their border
// 120 us (against 114), four states a lane and eight compute warps 121 us (against 103).
//
// One run is a whole sequence, or, where sequences times channel tiles leave
// SMs idle, a chunk of it (three launches): what every chunk adds to the state
// and the sum of its step sizes (the same kernel without c, y and z; the last
// chunks are left out), the states between the chunks, and the chunks
// themselves from those.
#include "gla_scan.cuh"

namespace gla {
namespace {

constexpr int kCompute = 128;  // threads of the recurrence
constexpr int kHelp = 128;     // threads of a helper group; group g of G serves stage g,
                               // through which the tiles g, g + G, ... pass
constexpr int threads_of(int groups) { return kCompute + groups * kHelp; }
// A whole sequence a block leaves one or two blocks a SM: a third helper group
// keeps the recurrence fed (8192 x 2048 x 16: 117 us with two, 109 with three, 114 with
// four, before the lanes' present order).  Chunks fill the SMs: two groups leave room
// for two blocks a SM (20001 packed tokens: one block 396 us, two 350).
// (Three groups' stages of fp32 rows do not fit at NS = 64.)
constexpr int kChunkGroups = 2;
template <typename IO, int NS> constexpr int whole_groups() {
  return sizeof(IO) == 4 && NS == 64 ? 2 : 3;
}
constexpr int kPairs = 1024;   // (token, channel) pairs of a tile
constexpr int kV = 8;          // adjacent channels of a token: a helper's pairs of a tile

// Named barriers 1 + g: stage g prepared; 1 + G + g: stage g used.  Each joins the
// compute warps and one helper group.
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kCompute + kHelp) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kCompute + kHelp) : "memory");
}

// What a chunked call keeps between its launches.
struct FwdSpace {
  float* h;    // [slots][D][NS]: what a chunk adds, then the state in front of it
  float* sum;  // [slots][D]: its step sizes
};

// The layout of a tile's shared memory.
template <typename IO, int NS, int G> struct Tile {
  static constexpr int LPC = NS / 8;              // lanes per channel
  static constexpr int CPW = 32 / LPC;            // channels per warp
  static constexpr int CT = kCompute / LPC;       // channels per block
  static constexpr int TT = kPairs / CT;          // tokens per tile
  static constexpr int NP = LPC > 1 ? 2 : 1;      // terms of a pair's sum over n
  static constexpr int HELD = 4 * NP / LPC;       // tokens (of 4) whose term a lane holds
  float2 d[G][TT * CT];                     // (delta, delta u); see dd_at
  float b[G][TT][NS], c[G][TT][NS];
  float y[G][NP][TT][CT];
  // rows as they come, each thread its own: of the tile in the stage, of the next
  // one of the group, and of those whose copies are in flight
  static constexpr int AHEAD = sizeof(IO) == 2 ? 2 : 1, RING = AHEAD + 2;
  Raw<IO, kV> u[G][RING][kHelp], dt[G][RING][kHelp], z[G][RING][kHelp];
  // Place of channel ch in a row of d: its 16-byte unit (two channels) is moved
  // within its 128 bytes so that the helpers' stores, 64 bytes apart, spread
  // over the banks.
  static __device__ __forceinline__ int dd_at(int ch) {
    const int unit = ch >> 1;
    return (unit ^ ((unit >> 3) & 3)) * 2 + (ch & 1);
  }
};

// Sums y[0 .. 4) over the lanes of a channel but one pair: afterwards a lane
// holds HELD of the four, from *first on, as one of NP terms.
template <int LPC, int CPW>
__device__ __forceinline__ void reduce_states(float (&y)[4], int q, int* first) {
  constexpr unsigned full = 0xffffffffu;
  *first = 0;
  if constexpr (LPC >= 4) {
    const bool up = (q & (LPC / 2)) != 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float give = up ? y[k] : y[k + 2], keep = up ? y[k + 2] : y[k];
      y[k] = keep + __shfl_xor_sync(full, give, CPW * LPC / 2);
    }
    *first = up ? 2 : 0;
  }
  if constexpr (LPC >= 8) {
    const bool up = (q & (LPC / 4)) != 0;
    const float give = up ? y[0] : y[1], keep = up ? y[1] : y[0];
    y[0] = keep + __shfl_xor_sync(full, give, CPW * LPC / 4);
    *first += up ? 1 : 0;
  }
}

// SUMS: the first of the three launches; else the scan itself, from init_state
// (chunk 0: one run per sequence) or from w.h.
template <typename IO, typename OUT, int NS, bool SUMS, int G>
__global__ void __launch_bounds__(threads_of(G), G == kChunkGroups ? 2 : 1)
scan_fwd_kernel(ScanArgs p, FwdSpace w, long long chunk) {
  if (!SUMS) after_previous();
  using L = Tile<IO, NS, G>;
  constexpr int LPC = L::LPC, CT = L::CT, TT = L::TT;
  extern __shared__ __align__(16) unsigned char smem[];
  L& s = *reinterpret_cast<L*>(smem);

  const int tiles = (p.D + CT - 1) / CT;
  const int d0 = (int)(blockIdx.x % tiles) * CT;
  const long long slot = blockIdx.x / tiles;
  Chunk k;
  if (chunk) {
    k = chunk_of_slot(p, slot, chunk);
    if (!k.ok || (SUMS && k.last)) return;
  } else {
    k.s = (int)slot;
    if (!seq_ok(p, k.s, threadIdx.x == 0, &k.t0, &k.t1)) return;
    k.last = true;
  }
  const int tiles_t = (int)((k.t1 - k.t0 + TT - 1) / TT);

  if (threadIdx.x < kCompute) {
    // lane bits: q's lowest, the channel's, q's others: reads by channel are the
    // same in lanes 1 apart and reads by q in lanes 2 apart, and either halves the
    // time of a read of 8 or 16 bytes a lane
    const int lane = threadIdx.x & 31, q = LPC == 1 ? 0 : (lane & 1) | (lane / L::CPW & ~1);
    const int lc = (threadIdx.x >> 5) * L::CPW + (LPC == 1 ? lane : lane / 2 % L::CPW);
    const int ch = min(d0 + lc, p.D - 1);
    auto load8 = [&](const float* from, f32x2 (&v)[4], float scale) {
      const float4* r = reinterpret_cast<const float4*>(from + (long long)ch * NS) + q * 2;
      const float4 x = r[0], y = r[1];
      v[0] = pack2(x.x * scale, x.y * scale);
      v[1] = pack2(x.z * scale, x.w * scale);
      v[2] = pack2(y.x * scale, y.y * scale);
      v[3] = pack2(y.z * scale, y.w * scale);
    };
    f32x2 a[4], h[4] = {};
    load8(p.a, a, kLog2e);
    if (!SUMS) {
      const float* from = chunk ? w.h + slot * p.D * NS
                                : p.init_state ? p.init_state + (long long)k.s * p.D * NS : nullptr;
      if (from) load8(from, h, 1.f);
    }
    const int at = L::dd_at(lc);
    float sum = 0.f;
    int buf = 0;
    for (int i = 0; i < tiles_t; ++i) {
      bar_sync(1 + buf);
      const float2* sd = &s.d[buf][at];
      const float* sb = &s.b[buf][0][q * 8];
      const float* sc = &s.c[buf][0][q * 8];
      // Token t's row of d, b, c, in registers from two tokens before its use;
      // its decays from one token before.  (The two rows read behind the tile's
      // last lie in the arrays behind; nothing comes of them.)
      struct Row {
        float2 d;
        f32x2 b[4], c[4];
      };
      auto fetch = [&](int t, Row& r) {
        r.d = sd[t * CT];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float4 v = reinterpret_cast<const float4*>(sb + t * NS)[m];
          r.b[2 * m] = pack2(v.x, v.y);
          r.b[2 * m + 1] = pack2(v.z, v.w);
          if (!SUMS) {
            const float4 x = reinterpret_cast<const float4*>(sc + t * NS)[m];
            r.c[2 * m] = pack2(x.x, x.y);
            r.c[2 * m + 1] = pack2(x.z, x.w);
          }
        }
      };
      Row r[4];  // token t in r[t % 4]
      f32x2 e[4];
      fetch(0, r[0]);
      fetch(1, r[1]);
#pragma unroll
      for (int m = 0; m < 4; ++m) e[m] = decay2<sizeof(IO) == 4>(mul2(both(r[0].d.x), a[m]));
#pragma unroll 1
      for (int t4 = 0; t4 < TT; t4 += 4) {
        float y[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          fetch(t4 + x + 2, r[(x + 2) % 4]);
          const Row& cur = r[x];
          const f32x2 dl = both(r[(x + 1) % 4].d.x), du = both(cur.d.y);
          f32x2 ys = {};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const f32x2 en = decay2<sizeof(IO) == 4>(mul2(dl, a[m]));
            h[m] = fma2(e[m], h[m], mul2(du, cur.b[m]));
            if (!SUMS) ys = m == 0 ? mul2(cur.c[0], h[0]) : fma2(cur.c[m], h[m], ys);
            e[m] = en;
          }
          if (SUMS) {
            sum += cur.d.x;
          } else {
            float y0, y1;
            unpack2(ys, &y0, &y1);
            y[x] = y0 + y1;
          }
        }
        if constexpr (!SUMS) {
          int first;
          reduce_states<LPC, L::CPW>(y, q, &first);
#pragma unroll
          for (int m = 0; m < L::HELD; ++m) s.y[buf][q & (L::NP - 1)][t4 + first + m][lc] = y[m];
        }
      }
      bar_arrive(1 + G + buf);
      buf = buf + 1 == G ? 0 : buf + 1;
    }
    if (d0 + lc < p.D) {
      float* to = SUMS ? w.h + slot * p.D * NS
                       : k.last && p.final_state ? p.final_state + (long long)k.s * p.D * NS : nullptr;
      if (to) {
        float4* r = reinterpret_cast<float4*>(to + (long long)ch * NS) + q * 2;
        float4 x, y;
        unpack2(h[0], &x.x, &x.y);
        unpack2(h[1], &x.z, &x.w);
        unpack2(h[2], &y.x, &y.y);
        unpack2(h[3], &y.z, &y.w);
        r[0] = x;
        r[1] = y;
      }
      if (SUMS && q == 0) w.sum[slot * p.D + ch] = sum;
    }
    return;
  }

  // the helper groups: a thread owns kV channels of one token of its tiles
  const int tid = (threadIdx.x - kCompute) % kHelp, g = (threadIdx.x - kCompute) / kHelp;
  constexpr int VPT = CT / kV;            // threads per token
  const int vt = tid / VPT, vc = (tid % VPT) * kV;
  const bool von = d0 + vc < p.D;
  f32x2 bias[kV / 2], skip[kV / 2];
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) {
    const int ch = d0 + vc + 2 * i;
    bias[i] = von && p.dt_bias ? pack2(__ldg(p.dt_bias + ch), __ldg(p.dt_bias + ch + 1)) : f32x2{};
    skip[i] = !SUMS && von && p.skip ? pack2(__ldg(p.skip + ch), __ldg(p.skip + ch + 1)) : f32x2{};
  }
  using R = Raw<IO, kV>;
  constexpr int BC = (TT * NS + kHelp - 1) / kHelp;  // b (and c) elements per thread and tile
  constexpr bool AHEAD = BC <= 4;                    // ... kept in registers a group's tile ahead
  constexpr int STEP = G * TT;                 // tokens from a group's tile to its next
  IO rb[AHEAD ? BC : 1], rc[AHEAD ? BC : 1];
  const long long row = k.t0 + g * TT + vt;
  const IO* pu = (const IO*)p.u + row * p.u_stride + d0 + vc;
  const IO* pd = (const IO*)p.dt + row * p.dt_stride + d0 + vc;
  const IO* pz = !SUMS && p.z ? (const IO*)p.z + row * p.z_stride + d0 + vc : nullptr;
  OUT* po = (OUT*)p.out + row * p.D + d0 + vc;
  const int left = (int)(k.t1 - k.t0);               // tokens of the run
  // this thread's elements of b and c: column tid % NS of the rows tid / NS, tid /
  // NS + kHelp / NS, ... of a tile
  constexpr int BROWS = kHelp / NS;
  const IO* pb = (const IO*)p.b + (k.t0 + g * TT + tid / NS) * p.b_stride + tid % NS;
  const IO* pc = (const IO*)p.c + (k.t0 + g * TT + tid / NS) * p.c_stride + tid % NS;
  int t_bc = g * TT + tid / NS;   // the first one's token
  auto copy = [](R* to, const IO* from) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(R) / 16; ++i)
      cp_async16(reinterpret_cast<char*>(to) + 16 * i, reinterpret_cast<const char*>(from) + 16 * i);
  };
  int put = 0, get = 0;           // ring places of the next tile to load and to prepare
  auto next = [](int i) { return i + 1 == L::RING ? 0 : i + 1; };
  int t_load = g * TT + vt;       // this thread's token in the next tile to load
  auto load = [&]() {             // always one group of copies, even of nothing
    if (t_load < left && von) {
      copy(&s.u[g][put][tid], pu);
      copy(&s.dt[g][put][tid], pd);
      if (!SUMS && p.z) copy(&s.z[g][put][tid], pz);
    }
    cp_commit();
    put = next(put);
    t_load += STEP;
    pu += STEP * p.u_stride;
    pd += STEP * p.dt_stride;
    if (!SUMS && p.z) pz += STEP * p.z_stride;
  };
  auto next_bc = [&]() {
    t_bc += STEP;
    pb += STEP * p.b_stride;
    pc += STEP * p.c_stride;
  };
  auto load_bc = [&]() {
    if constexpr (AHEAD) {
#pragma unroll
      for (int e = 0; e < BC; ++e) {
        rb[e] = rc[e] = from_f32<IO>(0.f);
        if (t_bc + e * BROWS < left) {
          rb[e] = pb[e * BROWS * p.b_stride];
          if (!SUMS) rc[e] = pc[e * BROWS * p.c_stride];
        }
      }
      next_bc();
    }
  };
  auto store_bc = [&]() {
    float* sb = &s.b[g][0][0];
    float* sc = &s.c[g][0][0];
    if constexpr (AHEAD) {
#pragma unroll
      for (int e = 0; e < BC; ++e) {
        const int x = tid + e * kHelp;
        if (TT * NS % kHelp != 0 && x >= TT * NS) break;
        sb[x] = to_f32(rb[e]);
        if (!SUMS) sc[x] = to_f32(rc[e]);
      }
    } else {
#pragma unroll 8
      for (int e = 0; e < BC; ++e) {
        const int x = tid + e * kHelp;
        const bool in = t_bc + e * BROWS < left;
        sb[x] = in ? to_f32(pb[e * BROWS * p.b_stride]) : 0.f;
        if (!SUMS) sc[x] = in ? to_f32(pc[e * BROWS * p.c_stride]) : 0.f;
      }
      next_bc();
    }
  };

  load_bc();
#pragma unroll
  for (int i = 0; i <= L::AHEAD; ++i) load();
  int last = 0;                   // ring place of the tile in the stage
  // one pass per tile of the group, and one to finish the last
  for (int tile = g; tile < tiles_t + G; tile += G) {
    const bool more = tile < tiles_t, prior = tile >= G;
    const int t = tile * TT + vt;
    // (delta, delta u) of the tile, before its stage is free
    f32x2 u[kV / 2], x[kV / 2];
#pragma unroll
    for (int j = 0; j < kV / 2; ++j) x[j] = u[j] = f32x2{};  // behind the run: decay 1, no drive
    if (more) {
      cp_wait<L::AHEAD>();
      if (t < left && von) {
        unpack_pairs<IO, kV>(s.u[g][get][tid], u);
        unpack_pairs<IO, kV>(s.dt[g][get][tid], x);
#pragma unroll
        for (int j = 0; j < kV / 2; ++j) {
          x[j] = add2(x[j], bias[j]);
          if (p.softplus) x[j] = softplus2<sizeof(IO) == 4>(x[j]);
          u[j] = mul2(x[j], u[j]);
        }
      }
    }
    f32x2 y[kV / 2];
    if (prior) {
      bar_sync(1 + G + g);
      if (!SUMS) {
#pragma unroll
        for (int m = 0; m < kV / 4; ++m) {
          const float4 v = *reinterpret_cast<const float4*>(&s.y[g][0][vt][vc + 4 * m]);
          y[2 * m] = pack2(v.x, v.y);
          y[2 * m + 1] = pack2(v.z, v.w);
          if (L::NP == 2) {
            const float4 v2 = *reinterpret_cast<const float4*>(&s.y[g][L::NP - 1][vt][vc + 4 * m]);
            y[2 * m] = add2(y[2 * m], pack2(v2.x, v2.y));
            y[2 * m + 1] = add2(y[2 * m + 1], pack2(v2.z, v2.w));
          }
        }
      }
    }
    if (more) {
      store_bc();
#pragma unroll
      for (int j = 0; j < kV / 2; ++j) {
        float d0v, d1v, u0, u1;
        unpack2(x[j], &d0v, &d1v);
        unpack2(u[j], &u0, &u1);
        *reinterpret_cast<float4*>(&s.d[g][vt * CT + L::dd_at(vc + 2 * j)]) =
            make_float4(d0v, u0, d1v, u1);
      }
      bar_arrive(1 + g);
      load_bc();
    }
    if (!SUMS && prior && t - STEP < left && von) {
      f32x2 z[kV / 2];
      float o[kV];
      unpack_pairs<IO, kV>(s.u[g][last][tid], u);
      if (p.z) unpack_pairs<IO, kV>(s.z[g][last][tid], z);
#pragma unroll
      for (int j = 0; j < kV / 2; ++j) {
        f32x2 v = fma2(skip[j], u[j], y[j]);
        if (p.z) v = mul2(v, mul2(z[j], sigmoid2(z[j])));
        unpack2(v, &o[2 * j], &o[2 * j + 1]);
      }
      store_raw<OUT, kV>(po, pack_as<OUT, kV>(o));
    }
    if (prior) po += STEP * (long long)p.D;
    last = get;
    get = next(get);
    if (more) load();
  }
  cp_wait<0>();
}

// The states in front of the chunks, and the final states of empty sequences.
__global__ void __launch_bounds__(128)
scan_fwd_chunks_kernel(ScanArgs p, FwdSpace w, long long chunk) {
  after_previous();
  const int quads = p.NS / 4;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long per = (long long)p.D * quads;
  if (i >= per * p.B) return;
  const int s = (int)(i / per);
  const long long in = i % per;
  long long lo, hi;
  if (!seq_ok(p, s, in == 0, &lo, &hi)) return;
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.init_state) run = reinterpret_cast<const float4*>(p.init_state)[(long long)s * per + in];
  if (lo == hi) {
    if (p.final_state) reinterpret_cast<float4*>(p.final_state)[(long long)s * per + in] = run;
    return;
  }
  float4 x = __ldg(reinterpret_cast<const float4*>(p.a) + in);
  x.x *= kLog2e; x.y *= kLog2e; x.z *= kLog2e; x.w *= kLog2e;
  // the last chunk's own sums were left out: its slot only receives a state
  const long long f = first_slot(p, s, chunk), n = (hi - lo + chunk - 1) / chunk;
  scan_chunks(reinterpret_cast<float4*>(w.h), w.sum, x, f, n - 1, per, in, p.D, (int)(in / quads),
              false, &run);
  reinterpret_cast<float4*>(w.h)[(f + n - 1) * per + in] = run;
}

template <typename IO, typename OUT, int NS, bool SUMS, int G>
cudaError_t launch_kernel(const ScanArgs& a, const FwdSpace& w, long long chunk, long long runs,
                          cudaStream_t stream) {
  constexpr int CT = Tile<IO, NS, G>::CT, smem = (int)sizeof(Tile<IO, NS, G>);
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  auto kernel = scan_fwd_kernel<IO, OUT, NS, SUMS, G>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel, smem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((long long)((a.D + CT - 1) / CT) * runs));
  if (!SUMS && chunk)
    return launch_after(kernel, grid, dim3(threads_of(G)), smem, stream, a, w, chunk);
  kernel<<<grid, threads_of(G), smem, stream>>>(a, w, chunk);
  return cudaGetLastError();
}

// About the time of a launch of `full` blocks of `len` tokens and `part` blocks of
// `rest` tokens at two blocks a SM, in tokens; a block that has a SM to itself takes
// two thirds, a start costs as much as 24 tokens.
long long span(long long full, long long len, long long part, long long rest) {
  constexpr long long kSlots = 2 * 152;
  len += 24;
  rest += 24;
  const long long waves = full / kSlots, over = full % kSlots, left = kSlots - over;
  const bool room = over + part <= kSlots / 2;
  if (over == 0) return waves * len + (part == 0 ? 0 : room ? rest * 2 / 3 : rest);
  const long long last = room ? len * 2 / 3 : len;  // the last wave's whole chunks
  if (part == 0) return waves * len + last;
  const long long beside = (part + left - 1) / left * rest;  // short ones in the slots left
  return waves * len + (beside < last ? last : beside < last + rest ? beside : last + rest);
}

// The chunk length of a call, 0 for whole sequences.  In units of a block's time
// for one token (about 0.05 us at NS = 16, a block a SM): whole sequences take the
// longest one times the waves of blocks; chunks take 1.7 times the work (the
// extra pass) spread over all SMs, and about 100 for two more launches.  A packed
// call's longest sequence is not known here: 2.5 times the mean.  Measured, D =
// 2048 and NS = 16, whole against best chunk: 4 x 2048 tokens 103 and 154 us, 2 x 2048
// 103 and 84, 1 x 2048 103 and 45, 1 x 512 29 and 19, three packed sequences of 20001
// tokens 708 and 347.
//
// Equal sequences: the length whose blocks fill their waves best.  1 x 2048 tokens: 224 45
// us, 256 50, 208 52, 320 60; 1 x 8192: 864 147 us, 896 152, 576 153, 1024 171, 768
// 193.  Packed ones: about four blocks a SM (two are resident); the last case in 1024 347 us,
// in 512 357, in 64 504, in 2048 397.  The constants are those of 16 states: with 64 the
// rule errs where it is close (1 x 5000 tokens of 1024 channels: 287 us, whole 254).
long long chunk_rule(int B, long long rows, int D, int NS, bool packed) {
  constexpr long long kSMs = 152;
  const long long tiles = ((long long)D * NS + 1023) / 1024, work = rows * tiles / kSMs;
  long long longest = (rows + B - 1) / B;
  if (packed && B > 1) longest = longest * 5 / 2 < rows ? longest * 5 / 2 : rows;
  const long long whole = (B * tiles + kSMs - 1) / kSMs * longest;
  if (work * 17 / 10 + 100 >= whole) return 0;
  long long chunk = 64;
  if (packed && B > 1) {
    while (chunk * 6 < work && chunk < 1024) chunk *= 2;  // nearest power of two to work / 4
    return chunk;
  }
  long long least = 0;
  for (long long c = 64; c <= 1024; c += 16) {
    const long long n = longest / c, rest = longest % c, blocks = B * tiles;
    const long long t = span(n * blocks, c, rest ? blocks : 0, rest) +
                        span((rest ? n : n - 1) * blocks, c, 0, 0) * 2 / 3;
    if (c == 64 || t < least) {
      least = t;
      chunk = c;
    }
  }
  return least * 2 + 40 >= whole ? 0 : chunk;  // (1 x 256 tokens: 15.8 us whole, 14.3 in chunks)
}

template <typename IO, typename OUT, int NS>
cudaError_t launch_typed(const ScanArgs& a, void* workspace, cudaStream_t stream) {
  const long long rows = a.cu_seqlens ? (long long)a.T : (long long)a.B * a.T;
  const long long chunk = rows > 0 ? chunk_rule(a.B, rows, a.D, NS, a.cu_seqlens != nullptr) : 0;
  if (chunk == 0)
    return launch_kernel<IO, OUT, NS, false, whole_groups<IO, NS>()>(a, FwdSpace{}, 0, a.B,
                                                                     stream);
  const long long slots = slots_of(a.B, rows, chunk);
  FwdSpace w;
  w.h = static_cast<float*>(workspace);
  w.sum = w.h + slots * a.D * NS;
  cudaError_t e = launch_kernel<IO, OUT, NS, true, kChunkGroups>(a, w, chunk, slots, stream);
  if (e != cudaSuccess) return e;
  const long long per = (long long)a.B * a.D * (NS / 4);
  e = launch_after(scan_fwd_chunks_kernel, dim3((unsigned)((per + 127) / 128)), dim3(128), 0,
                   stream, a, w, chunk);
  return e != cudaSuccess
             ? e
             : launch_kernel<IO, OUT, NS, false, kChunkGroups>(a, w, chunk, slots, stream);
}

template <typename IO, typename OUT>
cudaError_t launch_io(const ScanArgs& a, void* workspace, cudaStream_t stream) {
  switch (a.NS) {
    case 8: return launch_typed<IO, OUT, 8>(a, workspace, stream);
    case 16: return launch_typed<IO, OUT, 16>(a, workspace, stream);
    case 32: return launch_typed<IO, OUT, 32>(a, workspace, stream);
    default: return launch_typed<IO, OUT, 64>(a, workspace, stream);
  }
}

}  // namespace

size_t scan_fwd_workspace(int B, long long rows, int D, int NS, bool packed) {
  const long long chunk = chunk_rule(B, rows, D, NS, packed);
  return chunk ? (size_t)slots_of(B, rows, chunk) * D * (NS + 1) * 4 : 0;
}

cudaError_t launch_scan_fwd(const ScanArgs& a, void* workspace, cudaStream_t stream) {
  if (a.fp32_io) return launch_io<float, float>(a, workspace, stream);
  if (a.fp32_out) return launch_io<__nv_bfloat16, float>(a, workspace, stream);
  return launch_io<__nv_bfloat16, __nv_bfloat16>(a, workspace, stream);
}

}  // namespace gla
