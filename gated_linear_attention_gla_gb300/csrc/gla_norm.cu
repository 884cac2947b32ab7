// gla_norm.cu -- what stands between two blocks, in one pass over each row:
//
//     p = norm(y) post_weight + post_bias      (norm: RMS, or layer norm)
//     s = res + scale p silu(z)
//     u = norm(s) weight + bias
//
// norm(x) = c / sqrt(mean(c^2) + eps), c = x or x - mean(x).  Everything between
// the loads and the two stores is fp32 (s is rounded where it is stored, u comes
// from the unrounded s); the mean square is of the centred values, which lie in
// registers, so nothing cancels.
//
// A group of threads owns a row, eight adjacent channels a thread and vector; the
// sums over the row are shuffles and one exchange through shared memory.
// Bound: HBM.
#include "gla_norm.cuh"

namespace gla {
namespace {

using namespace norm;

template <typename T, typename RT, typename OT, int K>
__global__ void norm_fwd_kernel(NormArgs a, int tpr, long long stride_rows) {
  extern __shared__ float red[];
  const Group g(tpr, red);
  long long row = (long long)blockIdx.x * g.count + g.index;
  for (; row < a.rows; row += stride_rows) {
    float s[K][kV];
    const RT* res = (const RT*)a.res + row * a.D;
    each<K>(g, a.D, [&](int k, int c) { load_f32<RT>(res + c, s[k]); }, s);
    if (a.y) {
      float y[K][kV];
      const T* yr = (const T*)a.y + row * a.y_stride;
      each<K>(g, a.D, [&](int k, int c) { load_f32<T>(yr + c, y[k]); }, y);
      Raw<T, kV> z[K];
      if (a.z) {
        const T* zr = (const T*)a.z + row * a.z_stride;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int c = g.column(k);
          z[k] = c < a.D ? load_raw<T, kV>(zr + c) : zero_raw<T, kV>();
        }
      }
      if (a.post_weight) {
        const float r = normalise<K>(g, a, y);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int c = g.column(k);
          if (c >= a.D) continue;
          float w[kV];
          load_vec(a.post_weight + c, w);
          float b[kV] = {};
          if (a.post_bias) load_vec(a.post_bias + c, b);
#pragma unroll
          for (int j = 0; j < kV; ++j) y[k][j] = fmaf(y[k][j] * r, w[j], b[j]);
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = g.column(k);
        if (c >= a.D) continue;
        if (a.z) {
          float zf[kV];
          unpack_as<T, kV>(z[k], zf);
#pragma unroll
          for (int j = 0; j < kV; ++j) y[k][j] *= silu(zf[j]);
        }
        float w[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) w[j] = 1.f;
        if (a.scale) load_vec(a.scale + c, w);
#pragma unroll
        for (int j = 0; j < kV; ++j) s[k][j] = fmaf(w[j], y[k][j], s[k][j]);
        if (a.res_out) store_raw<RT, kV>((RT*)a.res_out + row * a.D + c, pack_as<RT, kV>(s[k]));
      }
    }
    if (a.out) {
      const float r = normalise<K>(g, a, s);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = g.column(k);
        if (c >= a.D) continue;
        float w[kV];
        load_vec(a.weight + c, w);
        float b[kV] = {};
        if (a.bias) load_vec(a.bias + c, b);
        float u[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) u[j] = fmaf(s[k][j] * r, w[j], b[j]);
        store_raw<OT, kV>((OT*)a.out + row * a.D + c, pack_as<OT, kV>(u));
      }
    }
  }
}

template <typename T, typename RT, typename OT>
cudaError_t run_fwd(const NormArgs& a, cudaStream_t stream) {
  const Shape s = fwd_shape(a.D);
  const long long blocks = (a.rows + s.groups - 1) / s.groups;
  const int threads = s.tpr * s.groups, smem = s.groups * kRedFloats * 4;
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)blocks, threads, smem, stream>>>(a, s.tpr, blocks * s.groups);
    return cudaGetLastError();
  };
  if (s.k == 1) return go(norm_fwd_kernel<T, RT, OT, 1>);
  return go(norm_fwd_kernel<T, RT, OT, 2>);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  if (a.fp32_io) return run_fwd<float, float, float>(a, stream);
  if (a.fp32_res) return a.fp32_out ? run_fwd<bf16, float, float>(a, stream)
                                    : run_fwd<bf16, float, bf16>(a, stream);
  return a.fp32_out ? run_fwd<bf16, bf16, float>(a, stream)
                    : run_fwd<bf16, bf16, bf16>(a, stream);
}

}  // namespace gla
