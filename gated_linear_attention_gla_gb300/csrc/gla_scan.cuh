// gla_scan.cuh -- what the forward and backward scan kernels share.
#pragma once

#include "gla_ssm.cuh"

namespace gla {

// The sum of y[k] over the LPC lanes of a channel, scattered: lane q ends up
// with 4 / LPC of the four sums (LPC = 2), one (4), or one shared by the lanes
// of a group (8, 16).  *first is the index of its first sum.
template <int LPC>
__device__ __forceinline__ void reduce4(float (&y)[4], int q, int* first) {
  constexpr unsigned full = 0xffffffffu;
  // halve the list: the upper lane of each pair keeps the upper half
  const bool up = (q & (LPC / 2)) != 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float give = up ? y[k] : y[k + 2];
    const float keep = up ? y[k + 2] : y[k];
    y[k] = keep + __shfl_xor_sync(full, give, LPC / 2);
  }
  *first = up ? 2 : 0;
  if constexpr (LPC >= 4) {
    const bool up2 = (q & (LPC / 4)) != 0;
    const float give = up2 ? y[0] : y[1];
    const float keep = up2 ? y[1] : y[0];
    y[0] = keep + __shfl_xor_sync(full, give, LPC / 4);
    *first += up2 ? 1 : 0;
#pragma unroll
    for (int off = LPC / 8; off > 0; off >>= 1) y[0] += __shfl_xor_sync(full, y[0], off);
  }
}

}  // namespace gla
