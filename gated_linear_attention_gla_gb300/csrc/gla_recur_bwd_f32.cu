// gla_recur_bwd_f32.cu -- instances of the recurrence's gradient kernel for fp32 rows.
#include "gla_recur_bwd.cuh"

namespace gla {
namespace recur {

cudaError_t bwd_f32(const RecurBwdArgs& b, const Split& p, const float* kept,
                     long long kept_rows, float* partial, cudaStream_t stream) {
  return b.f.decay ? bwd_typed<float, true>(b, p, kept, kept_rows, partial, stream)
                   : bwd_typed<float, false>(b, p, kept, kept_rows, partial, stream);
}

}  // namespace recur
}  // namespace gla
