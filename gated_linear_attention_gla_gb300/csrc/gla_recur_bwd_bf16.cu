// gla_recur_bwd_bf16.cu -- instances of the recurrence's gradient kernel for bf16 rows.
#include "gla_recur_bwd.cuh"

namespace gla {
namespace recur {

cudaError_t bwd_bf16(const RecurBwdArgs& b, const Split& p, const float* kept,
                     long long kept_rows, float* partial, cudaStream_t stream) {
  return b.f.decay ? bwd_typed<__nv_bfloat16, true>(b, p, kept, kept_rows, partial, stream)
                   : bwd_typed<__nv_bfloat16, false>(b, p, kept, kept_rows, partial, stream);
}

}  // namespace recur
}  // namespace gla
