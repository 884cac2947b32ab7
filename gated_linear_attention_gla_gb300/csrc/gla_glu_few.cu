// gla_glu_few.cu -- the gated feed-forward projections of few rows (tokens of a decode step):
// the weights stream through once and bound the time, so they are the product's long side.
//
// A block takes 64 rows of Wg and the same 64 of Wu as the 128 rows of A and all N tokens (rounded up to 16) as B:
// lanes of the accumulator are the features, columns the tokens, and a stage of 64 along K is 16 KB of
// weights for at most 32 KB of tokens out of L2.  Where F has fewer such tiles than the GPU
// SMs, the blocks of a cluster share K and sum their accumulators through distributed
// shared memory, in block order.  g and u of a feature lie 64 lanes apart; the
// accumulators go through shared memory, from where the product leaves in rows of the output.
//
// Bound: HBM (the weights).  8 rows x 2048 x 8192 13.5 to 17.3 us by the GPU where kernels follow one
// another, 5.0 to 3.9 TB/s; x 4096 x 12288 34.6 us, 5.8 TB/s.
#include "gla_glu.cuh"

namespace gla {
namespace glu {
namespace {

constexpr int kThreads = 192;    // warps 0..3: accumulators, 4: producer, 5: issuer
constexpr int kFeatures = 64;    // of a block
constexpr int kLanes = 2 * kFeatures;  // rows of A
constexpr uint32_t kA = kLanes * kK * 2;
constexpr int kMaxStages = 10;
constexpr int kMaxSplit = 8;
constexpr int kPitch = kLanes + 4;  // floats between tokens of the accumulators in shared memory

struct FewParams {
  CUtensorMap x, wg, wu;
  void* out;
  int R, F, blocks_k;   // blocks of kK along K
  int N, stages;
  unsigned* status;
  uint64_t wait_ns;
};

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                         int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ float2 load_remote(const float* local, uint32_t rank) {
  uint32_t at;
  float2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

template <typename OT>
__global__ void __launch_bounds__(kThreads, 1) glu_few_kernel(const __grid_constant__ FewParams p,
                                                              int split) {
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t tmem_at;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = split > 1 ? (int)cta_rank() : 0;
  const int f0 = blockIdx.x / split * kFeatures;
  const int per = (p.blocks_k + split - 1) / split;
  const int k0 = rank * per, k1 = k0 + per < p.blocks_k ? k0 + per : p.blocks_k;
  const uint32_t stage_bytes = kA + (uint32_t)p.N * 128;
  const uint32_t cols = p.N <= 32 ? 32 : p.N <= 64 ? 64 : p.N <= 128 ? 128 : 256;
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&tmem_at, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  after_previous();
  start_next();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return wait_for(bar, parity, p.wait_ns, &abort_flag, p.status);
  };
  bool ok = true;
  if (warp == 4 && lane == 0) {
    int it = 0;
    for (int kb = k0; kb < k1; ++kb, ++it) {
      const int s = it % p.stages;
      if (it >= p.stages && !wait(&empty[s], (it / p.stages - 1) & 1)) break;
      mbar_arrive_expect_tx(&full[s], kA + p.N * 128);
      const uint32_t at = smem_u32(smem) + s * stage_bytes;
      load_box(at, &p.wg, &full[s], kb * kK, f0);
      load_box(at + kA / 2, &p.wu, &full[s], kb * kK, f0);
      load_box(at + kA, &p.x, &full[s], kb * kK, 0);
    }
    for (int i = it > p.stages ? it - p.stages : 0; i < it; ++i)  // every copy lands
      (void)mbar_wait_bounded(&full[i % p.stages], (i / p.stages) & 1, kDefaultWaitLimitNs);
  } else if (warp == 5) {
    const uint32_t idesc = idesc_bf16(kLanes, p.N, false, false);
    int it = 0;
    for (int kb = k0; kb < k1; ++kb, ++it) {
      const int s = it % p.stages;
      if (!__all_sync(0xffffffffu, wait(&full[s], (it / p.stages) & 1))) break;
      tc_fence_after();
      if (elect_one_sync()) {
        const uint32_t at = smem_u32(smem) + s * stage_bytes;
        const uint64_t da = sdesc_sw128(at, 0, 1024), db = sdesc_sw128(at + kA, 0, 1024);
#pragma unroll
        for (int k = 0; k < kK / 16; ++k)
          mma_bf16(tmem, desc_add(da, 32 * k), desc_add(db, 32 * k), idesc, it > 0 || k > 0);
        mma_commit(&empty[s]);
      }
      __syncwarp();
    }
    if (elect_one_sync()) mma_commit(&done);
    __syncwarp();
    ok = mbar_wait_bounded(&done, 0u, kDefaultWaitLimitNs);
  }
  ok = __syncthreads_and(ok && !abort_flag);  // products and copies are done: the stages are free
  tc_fence_after();
  // [token][lane]
  float* acc = reinterpret_cast<float*>(smem);
  if (ok && warp < 4) {
    const bool any = k1 > k0;
#pragma unroll 1
    for (int c = 0; c < p.N; c += 16) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(tmem + ((uint32_t)warp << 21) + c, r);
      tmem_ld_wait_x16(r);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        acc[(c + j) * kPitch + warp * 32 + lane] = any ? __uint_as_float(r[j]) : 0.f;
    }
    tc_fence_before();
  }
  if (split > 1) cluster_barrier();
  else __syncthreads();
  if (ok) {
    // two features a lane, the cluster's blocks take turns at the tokens
    const int f = 2 * lane;
    if (f0 + f < p.F) {
      for (int n = rank + warp * split; n < p.R; n += kThreads / 32 * split) {
        float2 g = make_float2(0.f, 0.f), u = g;
        const float* row = acc + n * kPitch + f;
        if (split == 1) {
          g = *reinterpret_cast<const float2*>(row);
          u = *reinterpret_cast<const float2*>(row + 64);
        } else {
          for (int q = 0; q < split; ++q) {
            g = add2(g, load_remote(row, q));
            u = add2(u, load_remote(row + 64, q));
          }
        }
        const float v[2] = {silu(g.x) * u.x, silu(g.y) * u.y};
        store_raw<OT, 2>((OT*)p.out + (long long)n * p.F + f0 + f, pack_as<OT, 2>(v));
      }
    }
  }
  if (split > 1) cluster_barrier();  // no block ends while another reads its sums
  if (warp == 5) tmem_dealloc(tmem, cols);
}

}  // namespace

cudaError_t launch_few(const GluArgs& a, cudaStream_t stream) {
  FewParams p{};
  p.out = a.out; p.R = a.rows; p.F = a.F; p.status = a.status;
  p.wait_ns = handoff_wait_limit_ns();
  p.blocks_k = tiles_of(a.D, kK);
  p.N = (a.rows + 15) / 16 * 16;
  // fewer than half of the SMs have a tile: several share its K (8 rows x 520 x 1352 4.2 us,
  // 5.6 us by a block a tile; of narrower tiles instead, 8 rows x 1024 x 4096 8.2 us, 6.7 us so)
  int split = 1;
  const int tiles = tiles_of(a.F, kFeatures);
  while (split < kMaxSplit && tiles * split * 2 <= 152 && split * 2 <= p.blocks_k) split *= 2;
  const int stage = (int)kA + p.N * 128;
  // more tiles than SMs: two blocks an SM, so that one's start and end lie under the other's
  // stream (8 rows x 4096 x 12288 34.6 us, with one block 47.6)
  p.stages = (tiles * split > 152 ? 104 : 208) * 1024 / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const int room = p.N * kPitch * 4 > p.stages * stage ? p.N * kPitch * 4 : p.stages * stage;
  if (!make_map(&p.x, a.x, a.D, a.rows, a.x_stride, p.N) ||
      !make_map(&p.wg, a.w_gate, a.D, a.F, a.D, kFeatures) ||
      !make_map(&p.wu, a.w_up, a.D, a.F, a.D, kFeatures))
    return cudaErrorInvalidValue;
  auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
    const cudaError_t e = allow_shared(kernel, 226 * 1024, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(tiles * split);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = room + 1024;
    c.stream = stream;
    c.attrs = attr;
    c.numAttrs = 2;
    return cudaLaunchKernelEx(&c, kernel, p, split);
  };
  static std::atomic<uint64_t> d0{0}, d1{0};
  return a.fp32_out ? go(glu_few_kernel<float>, d0) : go(glu_few_kernel<__nv_bfloat16>, d1);
}

}  // namespace glu
}  // namespace gla
