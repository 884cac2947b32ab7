// gla_norm.cu -- what stands between two blocks, in one pass over each row:
//
//     p = norm(y) post_weight + post_bias      (norm: RMS, or layer norm)
//     s = res + scale p silu(z)
//     u = norm(s) weight + bias
//
// norm(x) = c / sqrt(mean(c^2) + eps), c = x or x - mean(x).  Everything between
// the loads and the two stores is fp32 (s is rounded where it is stored, u comes
// from the unrounded s); layer norm's variance is of the centred values, which lie in registers, or of
// rows whose mean is small enough the mean square less the mean's (gla_norm.cuh).
//
// A group of threads owns a row, eight adjacent channels a thread and vector, and walks
// over rows, two at a time where there are many, with its parameters in registers and
// the next rows on their way into shared memory; the sums over the rows are shuffles
// and one exchange through shared memory.
// Bound: HBM.  16384 x 2048 with fp32 residuals 85 to 88 us, 5.4 TB/s; issue 40 %.
#include "gla_norm.cuh"

namespace gla {
namespace {

using namespace norm;

// R: rows at a time; BIAS: with post_bias or bias
template <typename T, typename RT, typename OT, int K, int R, bool BIAS>
__global__ void __launch_bounds__(512, 1)
norm_fwd_kernel(NormArgs a, int tpr, int stages) {
  extern __shared__ __align__(16) unsigned char shared[];
  const Group g(tpr, (float*)shared);
  after_previous();
  start_next();
  constexpr int kY = kPieces<RT>, kZ = kY + kPieces<T>;  // pieces behind res
  Ring<K> ring(shared + g.count * kRedFloats * 4, R, kZ + kPieces<T>, stages);
  Param<K> post, post_b, scale, weight, bias;
  post.init(g, a.D, a.post_weight, 1.f);
  scale.init(g, a.D, a.scale, 1.f);
  weight.init(g, a.D, a.weight, 1.f);
  if (BIAS) {
    post_b.init(g, a.D, a.post_bias, 0.f);
    bias.init(g, a.D, a.bias, 0.f);
  }
  const long long hop = (long long)gridDim.x * g.count * R;
  auto fetch = [&](long long row, int slot) {
    if constexpr (K == 1) {
      const int c = g.column(0);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (row + i < a.rows && c < a.D) {
          ring.copy(slot, i, 0, (const RT*)a.res + (row + i) * a.D + c);
          if (a.y) ring.copy(slot, i, kY, (const T*)a.y + (row + i) * a.y_stride + c);
          if (a.z) ring.copy(slot, i, kZ, (const T*)a.z + (row + i) * a.z_stride + c);
        }
      }
      cp_commit();
    }
  };
  long long row = ((long long)blockIdx.x * g.count + g.index) * R;
  for (int i = 0; i < stages - 1; ++i) fetch(row + i * hop, i);
  for (; row < a.rows; row += hop, ring.next()) {
    fetch(row + (stages - 1) * hop, ring.ahead());
    ring.wait();
    const int rows = R == 1 || row + 1 >= a.rows ? 1 : 2;
    auto has = [&](int i, int k) { return g.column(k) < a.D && i < rows; };
    Vec s[R][K];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k)
        s[i][k] = has(i, k)
                      ? ring.read(i, 0, (const RT*)a.res + (row + i) * a.D + g.column(k))
                      : vec_of(0.f);
    if (a.y) {
      Vec y[R][K];
      float r[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        r[i] = 1.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
          y[i][k] = has(i, k)
                        ? ring.read(i, kY, (const T*)a.y + (row + i) * a.y_stride + g.column(k))
                        : vec_of(0.f);
      }
      if (a.post_weight) normalise<K, R>(g, a, y, r, rows);
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int c = g.column(k);
          if (K > 1 && c >= a.D) continue;
          const Vec w = post.at(c), o = BIAS ? post_b.at(c) : w;
          Vec sc = scale.at(c);
          if (a.z) {
            const Vec z = has(i, k) ? ring.read(i, kZ, (const T*)a.z + (row + i) * a.z_stride + c)
                                    : vec_of(0.f);
#pragma unroll
            GLA_PAIRS sc.v[j] = mul2(sc.v[j], mul2(z.v[j], sigmoid2(z.v[j])));
          }
#pragma unroll
          GLA_PAIRS {
            const f32x2 n = mul2(y[i][k].v[j], both(r[i]));
            const f32x2 p = BIAS ? fma2(n, w.v[j], o.v[j]) : mul2(n, w.v[j]);
            s[i][k].v[j] = fma2(sc.v[j], p, s[i][k].v[j]);
          }
          if (a.res_out && has(i, k)) store_vec((RT*)a.res_out + (row + i) * a.D + c, s[i][k]);
        }
      }
    }
    if (a.out) {
      float r[R];
      normalise<K, R>(g, a, s, r, rows);
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int c = g.column(k);
          if (K > 1 && c >= a.D) continue;
          const Vec w = weight.at(c), o = BIAS ? bias.at(c) : w;
          Vec u;
#pragma unroll
          GLA_PAIRS {
            const f32x2 n = mul2(s[i][k].v[j], both(r[i]));
            u.v[j] = BIAS ? fma2(n, w.v[j], o.v[j]) : mul2(n, w.v[j]);
          }
          if (has(i, k)) store_vec((OT*)a.out + (row + i) * a.D + c, u);
        }
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
  const int other = s.groups * kRedFloats * 4;
  const long long hold = 152ll * blocks;
  auto go = [&](auto kernel, int R, std::atomic<uint64_t>& done) {
    const int pieces = R * (kPieces<RT> + 2 * kPieces<T>);
    const int stages = s.k == 1 ? ring_stages(pieces, threads, other, blocks) : 1;
    const int smem = other + (s.k == 1 ? stages * pieces * 16 * threads : 0);
    const long long need = ((long long)a.rows + s.groups * R - 1) / (s.groups * R);
    const cudaError_t e = allow_shared(kernel, 227 * 1024, done);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3((unsigned)(need < hold ? need : hold)), dim3(threads), smem,
                        stream, a, s.tpr, stages);
  };
  static std::atomic<uint64_t> d[6];
  const bool bias = a.post_bias || a.bias;
  if (s.k == 2)
    return bias ? go(norm_fwd_kernel<T, RT, OT, 2, 1, true>, 1, d[0])
                : go(norm_fwd_kernel<T, RT, OT, 2, 1, false>, 1, d[1]);
  // one row at a time where that fills no more than the GPU once (16 rows x 2048 2.0 us, 2.6 by twos;
  // 8192 rows 33.9 us, 30.8 by twos)
  if (a.rows <= hold * s.groups)
    return bias ? go(norm_fwd_kernel<T, RT, OT, 1, 1, true>, 1, d[2])
                : go(norm_fwd_kernel<T, RT, OT, 1, 1, false>, 1, d[3]);
  return bias ? go(norm_fwd_kernel<T, RT, OT, 1, 2, true>, 2, d[4])
              : go(norm_fwd_kernel<T, RT, OT, 1, 2, false>, 2, d[5]);
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
