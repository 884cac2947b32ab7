// gla_recur_bwd.cu -- the gradient of the gated linear recurrence, from its inputs alone.
// With e_t = dL/dh_t, s = sigmoid, and k = -dm / d(log a) = a^2 / m | a:
//     e_t = dy_t silu(z_t) + a_{t+1} e_{t+1}          (d_final behind the last token)
//     c_t = a h_{t-1} - k s(i) x,                      d(log a)_t = e_t c_t
//     dx = e m s(i),   di = e m x s(i) (1 - s(i)),     dz = dy h silu'(z)
//     df = e c log a (1 - s(f))  (without decay: e c (1 - s(f))),   d_decay = sum e c s(f)
//     d_init = a_0 e_0
// Two launches.  The forward kernel walks x, f and i once and keeps the state in
// front of every kKeep = 4 tokens; then the same split of the token axis
// (gla_recur.cuh) runs over e from the end.  A run is those 4 tokens: its states come again from the kept
// one, everything else that does not depend on e is reduced to factors of it in
// registers (each gradient is e times one number), and the map (Q_t, K_t) of e over the
// run is composed as in the forward.  d_decay: sums in registers over a thread's tokens, partials per
// block, summed in block order by a third launch.  No atomics.
// What takes the time: the wait for the states between a run's two halves, whose factors leave no registers
// for another run in between (issue 61 %, DRAM 47 %).
// 8192 x 2048 with three gates 103 us, 2.9 TB/s of what has to be moved; fp32 rows 143 us, 4.2 TB/s.
#include "gla_recur.cuh"

namespace gla {
namespace recur {
namespace {

// Sums the blocks' partials in block order: 32 channels a block.
__global__ void __launch_bounds__(1024)
decay_sum_kernel(float* d_decay, const float* partial, long long parts, int D) {
  after_previous();
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float t = 0.f;
  if (c < D)
    for (long long k = threadIdx.y; k < parts; k += 32) t += partial[k * D + c];
  part[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    for (int k = 1; k < 32; ++k) t += part[k][threadIdx.x];
    d_decay[c] = t;
  }
}

size_t kept_floats(const Split& p, int D) {
  const long long rows = (p.rows + kKeep - 1) / kKeep;
  return (size_t)(p.groups * rows * D + 63) / 64 * 64;
}

}  // namespace
}  // namespace recur

size_t recur_bwd_workspace(int B, long long rows, int D, bool packed) {
  using namespace recur;
  if (B <= 0) return 0;
  const Split p = split(B, (int)(packed ? rows : rows / B), D, packed, kKeep, kBwdWarps, kBwdBlocks);
  return (kept_floats(p, D) + (size_t)p.groups * p.cluster * D) * 4;
}

cudaError_t launch_recur_bwd(const RecurBwdArgs& b, void* workspace, cudaStream_t stream) {
  using namespace recur;
  const RecurArgs& a = b.f;
  if (a.B == 0)  // no sequences, no rows
    return b.d_decay ? cudaMemsetAsync(b.d_decay, 0, (size_t)a.D * 4, stream) : cudaSuccess;
  const Split p = split(a.B, a.T, a.D, a.cu_seqlens != nullptr, kKeep, kBwdWarps, kBwdBlocks);
  float* kept = static_cast<float*>(workspace);
  float* partial = kept + kept_floats(p, a.D);
  const long long kept_rows = (p.rows + kKeep - 1) / kKeep;
  cudaError_t e = a.fp32_io ? keep_f32(a, kept, kept_rows, stream) : keep_bf16(a, kept, kept_rows, stream);
  if (e != cudaSuccess) return e;
  e = a.fp32_io ? bwd_f32(b, p, kept, kept_rows, partial, stream)
                : bwd_bf16(b, p, kept, kept_rows, partial, stream);
  if (e != cudaSuccess || !b.d_decay) return e;
  return launch_after(decay_sum_kernel, dim3((a.D + 31) / 32), dim3(32, 32), 0, stream, b.d_decay,
                      (const float*)partial, p.groups * p.cluster, a.D);
}

}  // namespace gla
