// gla_glu.cuh -- what the kernels of the gated feed-forward projections share.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "gla_ssm.cuh"
#include "gla_sm100.cuh"

namespace gla {
namespace glu {

using namespace sm100;

constexpr int kK = 64;  // along K per stage (128 bytes of bf16)

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Waits for a phase of a barrier, for at most limit_ns of wall time; false: it ran out, or
// another role of the block has given up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                         volatile int* abort_flag, unsigned* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      atomicOr(status, kDevTimeout);
      return false;
    }
  }
  return true;
}

// ------------------------------------------------------------------ host side
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// bf16 [rows][cols], `stride` elements between rows; boxes of 64 columns x box_rows.
inline bool make_map(CUtensorMap* map, const void* base, long long cols, long long rows,
                     long long stride, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int tiles_of(long long n, int by) { return (int)((n + by - 1) / by); }

// The projections of at most kFewRows rows (gla_glu_few.cu; 128 rows x 2048 x 8192 16.0 us there and
// 18.0 us by tiles of 256 rows, x 520 x 1352 6.6 and 8.9 us; 192 rows 19.1 and 18.0 us).  Tiles of 256 rows
// cost the same for all of 129 to 256 rows, 18.4 to 18.8 us, of 257 to 512 25.1 to 25.9.
constexpr int kFewRows = 128;
cudaError_t launch_few(const GluArgs& a, cudaStream_t stream);

}  // namespace glu
}  // namespace gla
