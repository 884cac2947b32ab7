// gla_glu.cu -- the gated feed-forward projections and their gradient on the 5th-generation
// tensor cores.
//
//     g = x Wg^T, u = x Wu^T, out = g s u,  s = 1 / (1 + exp(-g))
//     dg = dout u s (1 + g (1 - s)), du = dout g s
//     dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// One kernel, a matrix product of 256 x 256 tiles by pairs of SMs (cta_group::2:
// either SM holds 128 rows of A and 128 of B, so a tile's operands cross into shared
// memory once), with three kinds of tiles:
//   kUp  out (or dg and du, with dout): A = x [256 rows], B = 128 rows of Wg (from the
//        pair's first SM) and the same 128 of Wu (from its second), so that one product
//        of N = 256 leaves g in columns 0..127 and u in 128..255 of the same
//        accumulator rows, and the epilogue has both in one thread.  g and u never
//        leave the chip.
//   kDx  A = dg, then du (the sum over K runs through both), B = Wg, Wu read along N
//   kDw  A = dg or du read along M, B = x read along N, K = the rows
// The backward is a kUp launch (dg, du into the workspace) and one launch of all kDx and kDw tiles.
// dg and du are rounded to bf16, once each: they are operands of the tensor cores' next products, beside x
// and the weights, which are bf16 too.  That puts dx and dw 0.0023 off their 64-bit values where one
// rounding of the results alone gives 0.0017, and so it is where fp32 results are asked for (their sums
// are fp32, of the rounded factors).  The other choice, two bf16 numbers for each, doubles these products:
// 20 R D F instead of 12.
//
// Roles (10 warps): 0..7 epilogue (thread = half of an accumulator row), 8 producer (TMA into a
// ring of 6 stages of 64 along K), 9 issuer (the first SM's alone).  The accumulators
// are two of 256 columns in tensor memory: a tile's epilogue overlaps the next tile's
// product.  Persistent: every pair takes each 76th tile.
// Every wait is bounded in wall time (gla_set_wait_limit_ns); one that runs out
// flags the status word, and the pair lets its copies and products land and ends.  Where one SM's block gave up
// the two producers may have stopped at different steps, and a barrier counts both SMs'
// bytes: they tell each other how far they came, the one behind catches up, and the
// first SM waits for the last steps.
// Bound: the tensor pipe, active in 96 % of the cycles of 8192 x 2048 x 8192: 267 to 284 us (2.06 to 1.94
// PFLOP/s) in series of some milliseconds, 316 to 319 us (1.74 PFLOP/s) in longer ones, where the power
// limit holds the clock near 1.5 GHz.  Gradients of 4096 rows likewise 470 to 510 and 515 to 520 us.
#include "gla_glu.cuh"

namespace gla {
namespace {

using namespace glu;

constexpr int kTile = 256;           // rows and columns of a pair's tile
constexpr int kHalf = 128;           // of one SM
constexpr int kStages = 6;
constexpr uint32_t kOperand = kHalf * kK * 2;          // 16 KB
constexpr uint32_t kStage = 2 * kOperand;
constexpr uint32_t kOffBar = kStages * kStage;
constexpr uint32_t kSmem = kOffBar + 256 + 1024;       // 1024: the window's alignment
constexpr int kEpilogue = 8;         // warps: two a lane quadrant, half of the columns each
constexpr int kThreads = 32 * (kEpilogue + 2);
constexpr uint32_t kCols = 512;                        // tensor memory: two accumulators

enum Bar { kFull = 0, kEmpty = kFull + kStages, kAccFull = kEmpty + kStages,
           kAccEmpty = kAccFull + 2, kDrain = kAccEmpty + 2, kNumBars };
static_assert(kNumBars * 8 + 16 <= 256, "barrier area");

struct GluParams {
  CUtensorMap x, wg, wu;      // kUp: boxes of 64 x 128 rows
  CUtensorMap dg, du;         // kDx's A: boxes of 64 x 128
  CUtensorMap dgm, dum, xm, wgm, wum;  // read along M or N: boxes of 64 x 64
  const __nv_bfloat16* d_out; // kUp of the backward, or null
  void* out;                  // kUp: out
  __nv_bfloat16 *dg_out, *du_out;
  void *dx, *dwg, *dwu;
  int R, D, F;
  int tiles, dx_tiles;        // of the launch; the first dx_tiles are kDx
  int tiles_m, tiles_n;       // kUp
  int dx_m, dx_width, dw_m, dw_n;  // tiles along the axes of kDx, kDw (dw_m: of one weight)
  int ahead;                  // kDw tiles that are as long as a kDx tile
  unsigned* status;
  uint64_t wait_ns;
};

// The address of the pair's first SM's copy of a shared variable.
__device__ __forceinline__ uint32_t first_sm(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
// A box into this SM's shared memory, counted on a barrier of the pair's first SM.
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, uint32_t bar, int c0,
                                         int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both SMs when the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void arrive_first_sm(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(first_sm(bar))
               : "memory");
}

// Two words of the pair's other block.
__device__ __forceinline__ void tell_other(volatile uint32_t* to, uint32_t rank, uint32_t x, uint32_t y) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(at)
      : "r"(smem_u32(const_cast<const uint32_t*>(to))), "r"(rank));
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}

enum Kind { kUp = 0, kDx = 1, kDw = 2 };
struct TileAt {
  int kind, m, n, seg;  // first row and column of the tile; seg: dg's or du's (kDw)
  int blocks;           // of kK along K
  int width;            // columns of the accumulator: 256, or 128 (kDx of few tiles)
};

// The i-th tile of a pair; false: it has no more.  The backward's second launch has two
// kinds of different length: the kDx tiles go around the pairs first; then the pairs that got one less
// take as many kDw tiles as one kDx tile is long, and the rest go around (4096 rows x
// 2048 x 8192: 862 steps of K a pair at best, 896 so, 960 without).
template <bool BWD2>
__device__ __forceinline__ bool tile_at(const GluParams& p, int pair, int pairs, int i, TileAt* a) {
  a->seg = 0;
  a->width = kTile;
  if (!BWD2) {
    const int t = pair + i * pairs;
    if (t >= p.tiles) return false;
    a->kind = kUp;
    a->m = t % p.tiles_m * kTile;
    a->n = t / p.tiles_m * kHalf;
    a->blocks = (p.D + kK - 1) / kK;
    return true;
  }
  const int dx = p.dx_tiles / pairs, more = p.dx_tiles % pairs;
  const int mine = dx + (pair < more);
  if (i < mine) {
    const int t = pair + i * pairs;
    a->kind = kDx;
    a->m = t % p.dx_m * kTile;
    a->n = t / p.dx_m * p.dx_width;
    a->width = p.dx_width;
    a->blocks = 2 * ((p.F + kK - 1) / kK);
    return true;
  }
  i -= mine;
  const int light = more ? pairs - more : 0, all = p.tiles - p.dx_tiles;
  int first = light * p.ahead;  // tiles that go to the light pairs
  if (first > all) first = all;
  int t = -1;
  if (light && pair >= more) {
    if (i < p.ahead) {
      t = (pair - more) + i * light;
      if (t >= first) return false;
    } else {
      i -= p.ahead;
    }
  }
  if (t < 0) t = first + pair + i * pairs;
  if (t >= all) return false;
  a->kind = kDw;
  a->n = t % p.dw_n * kTile;
  t /= p.dw_n;
  a->seg = t / p.dw_m;
  a->m = t % p.dw_m * kTile;
  a->blocks = (p.R + kK - 1) / kK;
  return true;
}

// Columns [c, c + 32) of an output row, from fp32.
template <typename OT>
__device__ __forceinline__ void store32(OT* row, int c, int cols, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    if (c + j < cols) {
      const float x[8] = {v[j], v[j + 1], v[j + 2], v[j + 3], v[j + 4], v[j + 5], v[j + 6], v[j + 7]};
      store_raw<OT, 8>(row + c + j, pack_as<OT, 8>(x));
    }
  }
}

// GRAD: kUp computes dg and du; BWD2: the tiles are kDx and kDw; OT: type of the outputs
template <bool BWD2, bool GRAD, typename OT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
glu_kernel(const __grid_constant__ GluParams p) {
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_at + 1);
  volatile uint32_t* other = tmem_at + 2;  // of the other SM: its producer's steps, whether it gave up
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars[kFull + i], 1);
      mbar_init(&bars[kEmpty + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[kAccFull + i], 1);
      mbar_init(&bars[kAccEmpty + i], 2 * kEpilogue);  // of either SM
    }
    mbar_init(&bars[kDrain], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kEpilogue + 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_at)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_barrier();
  const uint32_t tmem = *tmem_at;
  after_previous();

  auto wait = [&](int bar, uint32_t parity) {
    return wait_for(&bars[bar], parity, p.wait_ns, abort_flag, p.status);
  };
  auto wait_warp = [&](int bar, uint32_t parity) {  // the whole warp's answer
    return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
  };

  // The producer: `it` steps of K have been issued, the next one is block kb of the pair's i-th tile.
  const bool feeds = warp == kEpilogue && lane == 0;
  uint32_t it = 0;
  int tile = 0, kb = 0;
  bool more = false;
  TileAt at;
  auto feed = [&] {
    const int s = it % kStages;
    if (rank == 0)
      mbar_arrive_expect_tx(&bars[kFull + s], at.width == kTile ? 2 * kStage : kStage + kOperand);
    const uint32_t bar = first_sm(&bars[kFull + s]);
    unsigned char* sa = smem + s * kStage;
    unsigned char* sb = sa + kOperand;
    if (!BWD2) {
      load_box(sa, &p.x, bar, kb * kK, at.m + rank * kHalf);
      load_box(sb, rank ? &p.wu : &p.wg, bar, kb * kK, at.n);
    } else if (at.kind == kDx) {
      const int half = at.blocks / 2, seg = kb >= half, k = (kb - seg * half) * kK;
      load_box(sa, seg ? &p.du : &p.dg, bar, k, at.m + rank * kHalf);
      const CUtensorMap* w = seg ? &p.wum : &p.wgm;
      load_box(sb, w, bar, at.n + rank * (at.width / 2), k);
      if (at.width == kTile) load_box(sb + kOperand / 2, w, bar, at.n + rank * kHalf + 64, k);
    } else {
      const CUtensorMap* d = at.seg ? &p.dum : &p.dgm;
      load_box(sa, d, bar, at.m + rank * kHalf, kb * kK);
      load_box(sa + kOperand / 2, d, bar, at.m + rank * kHalf + 64, kb * kK);
      load_box(sb, &p.xm, bar, at.n + rank * kHalf, kb * kK);
      load_box(sb + kOperand / 2, &p.xm, bar, at.n + rank * kHalf + 64, kb * kK);
    }
    ++it;
    if (++kb == at.blocks) {
      kb = 0;
      more = tile_at<BWD2>(p, pair, pairs, ++tile, &at);
    }
  };

  if (feeds) {
    // ------------------------------------------------------------ producer
    more = tile_at<BWD2>(p, pair, pairs, 0, &at);
    while (more && (it < kStages || wait(kEmpty + it % kStages, (it / kStages - 1) & 1))) feed();
  } else if (warp == kEpilogue + 1 && rank == 0) {
    // ------------------------------------------------------------ issuer
    uint32_t it = 0, n = 0;
    bool ok = true;
    TileAt a;
    for (; ok && tile_at<BWD2>(p, pair, pairs, n, &a); ++n) {
      const bool a_mn = a.kind == kDw, b_mn = a.kind != kUp;
      const uint32_t idesc = idesc_bf16(kTile, a.width, false, false) | (a_mn ? 1u << 15 : 0u) |
                             (b_mn ? 1u << 16 : 0u);
      // along K per 16: 32 bytes of a 128-byte row, or 16 rows of 128 bytes
      const uint32_t step_a = a_mn ? 2048 : 32, step_b = b_mn ? 2048 : 32;
      const uint32_t d = tmem + (n & 1) * kTile;
      if (n >= 2 && !wait_warp(kAccEmpty + (n & 1), (n / 2 - 1) & 1)) break;
      tc_fence_after();
      for (int kb = 0; kb < a.blocks; ++kb, ++it) {
        const int s = it % kStages;
        if (!wait_warp(kFull + s, (it / kStages) & 1)) { ok = false; break; }
        tc_fence_after();
        if (elect_one_sync()) {
          const uint32_t at = smem_u32(smem + s * kStage);
          const uint64_t da = sdesc_sw128(at, kOperand / 2, 1024);
          const uint64_t db = sdesc_sw128(at + kOperand, kOperand / 2, 1024);
#pragma unroll
          for (int k = 0; k < kK / 16; ++k)
            mma_pair(d, desc_add(da, k * step_a), desc_add(db, k * step_b), idesc,
                     kb > 0 || k > 0);
          commit_pair(&bars[kEmpty + s]);
        }
        __syncwarp();
      }
      if (ok && elect_one_sync()) commit_pair(&bars[kAccFull + (n & 1)]);
      __syncwarp();
    }
    if (elect_one_sync()) {
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
              smem_u32(&bars[kDrain]))
          : "memory");
    }
    __syncwarp();
    (void)mbar_wait_bounded(&bars[kDrain], 0u, kDefaultWaitLimitNs);
  } else if (warp < kEpilogue) {
    // ------------------------------------------------------------ epilogue
    uint32_t n = 0;
    TileAt a;
    const int quad = warp & 3, half = warp >> 2;
    for (; tile_at<BWD2>(p, pair, pairs, n, &a); ++n) {
      const uint32_t acc = tmem + (n & 1) * kTile + ((uint32_t)quad << 21);
      const int row = a.m + rank * kHalf + quad * 32 + lane;
      if constexpr (!BWD2) {
        const bool on = row < p.R;
        const long long at = (long long)row * p.F;
        // dout a chunk ahead: the first one comes while the product runs
        Raw<__nv_bfloat16, 8> h[4];
        auto fetch = [&](int c) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = on && c + 8 * j < p.F ? load_raw<__nv_bfloat16, 8>(p.d_out + at + c + 8 * j)
                                         : zero_raw<__nv_bfloat16, 8>();
        };
        const int c0 = half * (kHalf / 2);
        if (GRAD) fetch(a.n + c0);
        if (!wait_warp(kAccFull + (n & 1), (n / 2) & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int c = c0; c < c0 + kHalf / 2; c += 32) {
          uint32_t gr[32], ur[32];
          tmem_ld_32x32b_x32(acc + c, gr);
          tmem_ld_32x32b_x32(acc + kHalf + c, ur);
          tmem_ld_wait_x32(gr);
          tmem_ld_wait_x32(ur);
          if constexpr (GRAD) {
            float dg[32], du[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const uint32_t hw = h[j / 8].w[j % 8 / 2];
              const float dh = __uint_as_float(j & 1 ? hw & 0xffff0000u : hw << 16);
              const float g = __uint_as_float(gr[j]), u = __uint_as_float(ur[j]);
              const float s = sigmoid(g), gs = g * s;
              du[j] = dh * gs;
              dg[j] = dh * u * fmaf(gs, 1.f - s, s);
            }
            if (c == c0) fetch(a.n + c + 32);
            if (on) {
              store32(p.dg_out + at, a.n + c, p.F, dg);
              store32(p.du_out + at, a.n + c, p.F, du);
            }
          } else {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = silu(__uint_as_float(gr[j])) * __uint_as_float(ur[j]);
            if (on) store32((OT*)p.out + at, a.n + c, p.F, v);
          }
          __syncwarp();  // the next loads are the whole warp's
        }
      } else {
        if (!wait_warp(kAccFull + (n & 1), (n / 2) & 1)) break;
        tc_fence_after();
        const int rows = a.kind == kDx ? p.R : p.F;
        OT* out = (OT*)(a.kind == kDx ? p.dx : a.seg ? p.dwu : p.dwg) + (long long)row * p.D;
        const bool on = row < rows;
        const int c0 = half * (a.width / 2);
#pragma unroll 1
        for (int c = c0; c < c0 + a.width / 2; c += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(acc + c, r);
          tmem_ld_wait_x32(r);
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          if (on) store32(out, a.n + c, p.D, v);
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first_sm(&bars[kAccEmpty + (n & 1)]);
    }
  }
  // the products issued are done, and unless a wait ran out so is every copy
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  start_next();
  if (feeds) tell_other(other, rank ^ 1, it, *abort_flag);
  cluster_barrier();
  if (*abort_flag || other[1]) {  // (the same in both blocks)
    // A producer is ahead by a ring at most, of stages whose products it knows to be done: the one
    // behind fills its half of them too, and then all copies of the ring land.
    if (feeds) {
      const uint32_t theirs = other[0];
      while (more && it < theirs) feed();
      if (rank == 0)
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
          (void)mbar_wait_bounded(&bars[kFull + i % kStages], (i / kStages) & 1,
                                  kDefaultWaitLimitNs);
    }
    cluster_barrier();
  }
  if (warp == kEpilogue + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols)
                 : "memory");
  }
}

template <bool BWD2, bool GRAD, typename OT>
cudaError_t launch(const GluParams& p, cudaStream_t stream, bool dependent) {
  static std::atomic<uint64_t> done{0};
  auto kernel = glu_kernel<BWD2, GRAD, OT>;
  cudaError_t e = allow_shared(kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  const int pairs = p.tiles < 76 ? p.tiles : 76;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(2 * pairs);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSmem;
  c.stream = stream;
  c.attrs = &attr;
  c.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, p);
}

bool up_params(const GluArgs& a, GluParams* p) {
  p->R = a.rows; p->D = a.D; p->F = a.F;
  p->tiles_m = tiles_of(a.rows, kTile);
  p->tiles_n = tiles_of(a.F, kHalf);
  p->tiles = p->tiles_m * p->tiles_n;
  p->status = a.status;
  p->wait_ns = handoff_wait_limit_ns();
  return make_map(&p->x, a.x, a.D, a.rows, a.x_stride, kHalf) &&
         make_map(&p->wg, a.w_gate, a.D, a.F, a.D, kHalf) &&
         make_map(&p->wu, a.w_up, a.D, a.F, a.D, kHalf);
}

}  // namespace

cudaError_t launch_glu_fwd(const GluArgs& a, cudaStream_t stream) {
  if (a.rows <= kFewRows) return launch_few(a, stream);
  GluParams p{};
  if (!up_params(a, &p)) return cudaErrorInvalidValue;
  p.out = a.out;
  return a.fp32_out ? launch<false, false, float>(p, stream, false)
                    : launch<false, false, __nv_bfloat16>(p, stream, false);
}

size_t glu_bwd_workspace(int rows, int D, int F) {
  return ((size_t)rows * F * 2 + 255) / 256 * 256 * 2;
}

cudaError_t launch_glu_bwd(const GluBwdArgs& b, void* workspace, cudaStream_t stream) {
  const GluArgs& a = b.f;
  const size_t gsz = a.fp32_out ? 4 : 2, w = (size_t)a.F * a.D * gsz;
  if (a.rows == 0) {
    const cudaError_t e = cudaMemsetAsync(b.dw_gate, 0, w, stream);
    return e != cudaSuccess ? e : cudaMemsetAsync(b.dw_up, 0, w, stream);
  }
  GluParams p{};
  if (!up_params(a, &p)) return cudaErrorInvalidValue;
  p.d_out = static_cast<const __nv_bfloat16*>(b.d_out);
  p.dg_out = static_cast<__nv_bfloat16*>(workspace);
  p.du_out = p.dg_out + glu_bwd_workspace(a.rows, a.D, a.F) / 4;
  cudaError_t e = launch<false, true, __nv_bfloat16>(p, stream, false);
  if (e != cudaSuccess) return e;
  p.dx = b.dx; p.dwg = b.dw_gate; p.dwu = b.dw_up;
  if (!make_map(&p.dg, p.dg_out, a.F, a.rows, a.F, kHalf) ||
      !make_map(&p.du, p.du_out, a.F, a.rows, a.F, kHalf) ||
      !make_map(&p.dgm, p.dg_out, a.F, a.rows, a.F, kK) ||
      !make_map(&p.dum, p.du_out, a.F, a.rows, a.F, kK) ||
      !make_map(&p.xm, a.x, a.D, a.rows, a.x_stride, kK) ||
      !make_map(&p.wgm, a.w_gate, a.D, a.F, a.D, kK) ||
      !make_map(&p.wum, a.w_up, a.D, a.F, a.D, kK))
    return cudaErrorInvalidValue;
  p.dx_m = tiles_of(a.rows, kTile);
  p.dw_m = tiles_of(a.F, kTile); p.dw_n = tiles_of(a.D, kTile);
  const int dw_tiles = 2 * p.dw_m * p.dw_n;
  // kDx tiles are the long ones: of half the width where there are pairs for them (gradients of
  // 777 rows x 520 x 1352 26.7 us, 31.6 us without)
  p.dx_width = p.dx_m * tiles_of(a.D, kHalf) + dw_tiles <= 76 ? kHalf : kTile;
  p.dx_tiles = p.dx_m * tiles_of(a.D, p.dx_width);
  p.tiles = p.dx_tiles + dw_tiles;
  const int dx_blocks = 2 * tiles_of(a.F, kK) * p.dx_width / kTile, dw_blocks = tiles_of(a.rows, kK);
  p.ahead = dx_blocks / dw_blocks;
  return a.fp32_out ? launch<true, false, float>(p, stream, true)
                    : launch<true, false, __nv_bfloat16>(p, stream, true);
}

}  // namespace gla
