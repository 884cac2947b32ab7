// gla_recur_fwd_f32.cu -- instances of the recurrence's prompt kernel for fp32 rows.
#include "gla_recur_fwd.cuh"

namespace gla {
namespace recur {

cudaError_t fwd_f32(const RecurArgs& a, cudaStream_t stream) {
  return a.decay ? fwd_typed<float, true>(a, stream) : fwd_typed<float, false>(a, stream);
}
cudaError_t keep_f32(const RecurArgs& a, float* kept, long long kept_rows, cudaStream_t stream) {
  return keep_typed<float>(a, kept, kept_rows, stream);
}

}  // namespace recur
}  // namespace gla
