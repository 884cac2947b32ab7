// gla_recur_fwd_bf16.cu -- instances of the recurrence's prompt kernel for bf16 rows.
#include "gla_recur_fwd.cuh"

namespace gla {
namespace recur {

cudaError_t fwd_bf16(const RecurArgs& a, cudaStream_t stream) {
  return a.decay ? fwd_typed<__nv_bfloat16, true>(a, stream) : fwd_typed<__nv_bfloat16, false>(a, stream);
}
cudaError_t keep_bf16(const RecurArgs& a, float* kept, long long kept_rows, cudaStream_t stream) {
  return keep_typed<__nv_bfloat16>(a, kept, kept_rows, stream);
}

}  // namespace recur
}  // namespace gla
