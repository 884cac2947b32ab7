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
// A group of threads owns a row, eight adjacent channels a thread and vector, and walks
// over rows with its parameters in registers and the next two rows on their way into
// shared memory; the sums over the row are shuffles and one exchange through shared
// memory.  Bound: HBM.
#include "gla_norm.cuh"

namespace gla {
namespace {

using namespace norm;

template <typename T, typename RT, typename OT, int K>
__global__ void __launch_bounds__(512, 1)
norm_fwd_kernel(NormArgs a, int tpr, int stages) {
  extern __shared__ __align__(16) unsigned char shared[];
  const Group g(tpr, (float*)shared);
  constexpr int kY = kPieces<RT>, kZ = kY + kPieces<T>;  // pieces behind res
  Ring<K> ring(shared + g.count * kRedFloats * 4, kZ + kPieces<T>, stages);
  Param<K> post, post_b, scale, weight, bias;
  post.init(g, a.D, a.post_weight, 1.f);
  post_b.init(g, a.D, a.post_bias, 0.f);
  scale.init(g, a.D, a.scale, 1.f);
  weight.init(g, a.D, a.weight, 1.f);
  bias.init(g, a.D, a.bias, 0.f);
  const long long hop = (long long)gridDim.x * g.count;
  auto fetch = [&](long long row, int slot) {
    if constexpr (K == 1) {
      const int c = g.column(0);
      if (row < a.rows && c < a.D) {
        ring.copy(slot, 0, (const RT*)a.res + row * a.D + c);
        if (a.y) ring.copy(slot, kY, (const T*)a.y + row * a.y_stride + c);
        if (a.z) ring.copy(slot, kZ, (const T*)a.z + row * a.z_stride + c);
      }
      cp_commit();
    }
  };
  long long row = (long long)blockIdx.x * g.count + g.index;
  for (int i = 0; i < stages - 1; ++i) fetch(row + i * hop, i);
  for (; row < a.rows; row += hop, ring.next()) {
    fetch(row + (stages - 1) * hop, ring.ahead());
    ring.wait();
    const RT* res = (const RT*)a.res + row * a.D;
    float s[K][kV];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (g.column(k) < a.D) ring.read(0, res + g.column(k), s[k]);
      else fill(s[k], 0.f);
    }
    if (a.y) {
      const T* yr = (const T*)a.y + row * a.y_stride;
      float y[K][kV];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (g.column(k) < a.D) ring.read(kY, yr + g.column(k), y[k]);
        else fill(y[k], 0.f);
      }
      const float r = a.post_weight ? normalise<K>(g, a, y) : 1.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = g.column(k);
        if (c >= a.D) continue;
        float w[kV], b[kV], sc[kV];
        post.at(c, w);
        post_b.at(c, b);
        scale.at(c, sc);
        if (a.z) {
          float z[kV];
          ring.read(kZ, (const T*)a.z + row * a.z_stride + c, z);
#pragma unroll
          for (int j = 0; j < kV; ++j) sc[j] *= silu(z[j]);
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) s[k][j] = fmaf(sc[j], fmaf(y[k][j] * r, w[j], b[j]), s[k][j]);
        if (a.res_out) store_raw<RT, kV>((RT*)a.res_out + row * a.D + c, pack_as<RT, kV>(s[k]));
      }
    }
    if (a.out) {
      const float r = normalise<K>(g, a, s);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = g.column(k);
        if (c >= a.D) continue;
        float w[kV], b[kV];
        weight.at(c, w);
        bias.at(c, b);
#pragma unroll
        for (int j = 0; j < kV; ++j) w[j] = fmaf(s[k][j] * r, w[j], b[j]);
        store_raw<OT, kV>((OT*)a.out + row * a.D + c, pack_as<OT, kV>(w));
      }
    }
  }
  cp_wait<0>();
}

template <typename T, typename RT, typename OT>
cudaError_t run_fwd(const NormArgs& a, cudaStream_t stream) {
  const Shape s = shape_of(a.D);
  const int threads = s.tpr * s.groups;
  const int blocks = threads <= 256 ? 2 : 1;  // an SM
  const int pieces = kPieces<RT> + 2 * kPieces<T>, other = s.groups * kRedFloats * 4;
  const int stages = s.k == 1 ? ring_stages(pieces, threads, other, blocks) : 1;
  const int smem = other + (s.k == 1 ? stages * pieces * 16 * threads : 0);
  const long long need = (a.rows + s.groups - 1) / s.groups, hold = 152ll * blocks;
  auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
    const cudaError_t e = allow_shared(kernel, 227 * 1024, done);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(need < hold ? need : hold), threads, smem, stream>>>(a, s.tpr, stages);
    return cudaGetLastError();
  };
  static std::atomic<uint64_t> d1{0}, d2{0};
  return s.k == 1 ? go(norm_fwd_kernel<T, RT, OT, 1>, d1) : go(norm_fwd_kernel<T, RT, OT, 2>, d2);
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
