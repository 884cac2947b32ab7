// gla_norm_bwd.cu -- the gradient of the norms, the gate and the residual sum between two
// blocks, from the forward's inputs alone.  With n = norm(s), p = norm(y) without
// their weights, q = p post_weight + post_bias, r the factors 1 / sqrt(mean + eps):
//     d_weight = sum du n,  d_bias = sum du
//     d = ds + r_s (dn - mean(dn) - n mean(dn n)),   dn = du weight     (mean(dn): layer norm)
//     d_res = d,  d_scale = sum d q silu(z),  dz = d scale q silu'(z)
//     dq = d scale silu(z),  d_post_weight = sum dq p,  d_post_bias = sum dq
//     dy = r_y (dp - mean(dp) - p mean(dp p)),       dp = dq post_weight
// One pass: a group of threads owns a row as in the forward (whose values it
// computes again) and walks over rows; the sums over rows stay with the thread that owns the
// column (in registers; in shared memory where a thread holds two vectors, whose
// eighty sums would not fit), are summed over a block's groups and written as one partial a
// block, which a second launch sums in block order.  No atomics: the same inputs
// give the same bits.
// Bound: HBM.
#include "gla_norm.cuh"

namespace gla {
namespace {

using namespace norm;

constexpr int kSums = 5;  // d_post_weight, d_post_bias, d_scale, d_weight, d_bias
constexpr int kThreads = 256;

// The sums of a thread's columns over the rows.
template <int K, bool SHARED> struct Sums {
  float v[SHARED ? 1 : kSums][SHARED ? 1 : K][SHARED ? 1 : kV];
  float* s;  // SHARED: element (i, k, j) at ((i K + k) kV + j) threads + thread
  __device__ void init(float* shared) {
    s = shared + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          if constexpr (SHARED) s[((i * K + k) * kV + j) * blockDim.x] = 0.f;
          else v[i][k][j] = 0.f;
        }
  }
  __device__ __forceinline__ void add(int i, int k, int j, float x, float y) {
    if constexpr (SHARED) {
      float& t = s[((i * K + k) * kV + j) * blockDim.x];
      t = fmaf(x, y, t);
    } else {
      v[i][k][j] = fmaf(x, y, v[i][k][j]);
    }
  }
  __device__ __forceinline__ float get(int i, int k, int j) const {
    if constexpr (SHARED) return s[((i * K + k) * kV + j) * blockDim.x];
    else return v[i][k][j];
  }
};

template <typename T, typename RT, typename GT, typename GRT, int K>
__global__ void __launch_bounds__(K == 1 ? 512 : 512)
norm_bwd_kernel(NormBwdArgs b, float* partial, int tpr) {
  start_next();
  extern __shared__ float shared[];
  constexpr bool kShared = K > 1;
  const NormArgs& a = b.f;
  const Group g(tpr, shared);
  Sums<K, kShared> sums;
  sums.init(shared + g.count * kRedFloats);
  for (long long row = (long long)blockIdx.x * g.count + g.index; row < a.rows;
       row += (long long)gridDim.x * g.count) {
    float s[K][kV], p[K][kV];
    Raw<T, kV> z[K], du[K];
    Raw<RT, kV> ds[K];
    float ry = 1.f;
    each<K>(g, a.D, [&](int k, int c) {
      load_f32<RT>((const RT*)a.res + row * a.D + c, s[k]);
    }, s);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = g.column(k);
      z[k] = a.z && c < a.D ? load_raw<T, kV>((const T*)a.z + row * a.z_stride + c)
                            : zero_raw<T, kV>();
      du[k] = b.d_out && c < a.D ? load_raw<T, kV>((const T*)b.d_out + row * a.D + c)
                                 : zero_raw<T, kV>();
      ds[k] = b.d_res_out && c < a.D ? load_raw<RT, kV>((const RT*)b.d_res_out + row * a.D + c)
                                     : zero_raw<RT, kV>();
    }
    if (a.y) {
      each<K>(g, a.D, [&](int k, int c) {
        load_f32<T>((const T*)a.y + row * a.y_stride + c, p[k]);
      }, p);
      if (a.post_weight) {
        ry = normalise<K>(g, a, p);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int j = 0; j < kV; ++j) p[k][j] *= ry;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j) p[k][j] = 0.f;
    }
    // q = p post_weight + post_bias, computed twice (again below) rather than held
    auto affine = [&](int k, float (&q)[kV]) {
      const int c = g.column(k);
#pragma unroll
      for (int j = 0; j < kV; ++j) q[j] = p[k][j];
      if (a.post_weight) {
        float w[kV], o[kV] = {};
        load_vec(a.post_weight + c, w);
        if (a.post_bias) load_vec(a.post_bias + c, o);
#pragma unroll
        for (int j = 0; j < kV; ++j) q[j] = fmaf(q[j], w[j], o[j]);
      }
    };
    auto scales = [&](int k, float (&w)[kV]) {
#pragma unroll
      for (int j = 0; j < kV; ++j) w[j] = 1.f;
      if (a.scale) load_vec(a.scale + g.column(k), w);
    };
    if (a.y && b.d_out) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (g.column(k) >= a.D) continue;
        float q[kV], w[kV];
        affine(k, q);
        scales(k, w);
        if (a.z) {
          float zf[kV];
          unpack_as<T, kV>(z[k], zf);
#pragma unroll
          for (int j = 0; j < kV; ++j) q[j] *= silu(zf[j]);
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) s[k][j] = fmaf(w[j], q[j], s[k][j]);
      }
    }
    // s becomes d = dL/ds
    if (b.d_out) {
      const float r = normalise<K>(g, a, s);
      float2 m = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (g.column(k) >= a.D) continue;
        float d[kV], w[kV];
        unpack_as<T, kV>(du[k], d);
        load_vec(a.weight + g.column(k), w);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const float n = s[k][j] * r;
          s[k][j] = n;
          sums.add(3, k, j, d[j], n);
          sums.add(4, k, j, d[j], 1.f);
          const float dn = d[j] * w[j];
          m.x = fmaf(dn, n, m.x);
          m.y += dn;
        }
      }
      m = g.sum(m);
      m.x *= a.inv_d;
      m.y = a.layer ? m.y * a.inv_d : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (g.column(k) >= a.D) continue;
        float d[kV], w[kV], e[kV];
        unpack_as<T, kV>(du[k], d);
        unpack_as<RT, kV>(ds[k], e);
        load_vec(a.weight + g.column(k), w);
#pragma unroll
        for (int j = 0; j < kV; ++j)
          s[k][j] = fmaf(r, fmaf(-s[k][j], m.x, fmaf(d[j], w[j], -m.y)), e[j]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) unpack_as<RT, kV>(ds[k], s[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (g.column(k) < a.D)
        store_raw<GRT, kV>((GRT*)b.d_res + row * a.D + g.column(k), pack_as<GRT, kV>(s[k]));
    if (!a.y) continue;
    // s becomes dp, then dy
    float2 m = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = g.column(k);
      if (c >= a.D) continue;
      float q[kV], w[kV], zf[kV];
      affine(k, q);
      scales(k, w);
      unpack_as<T, kV>(z[k], zf);
      float dz[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const float sig = a.z ? sigmoid(zf[j]) : 1.f;
        const float gate = a.z ? zf[j] * sig : 1.f;
        sums.add(2, k, j, s[k][j], q[j] * gate);
        const float d = s[k][j] * w[j];
        dz[j] = d * q[j] * fmaf(gate, 1.f - sig, sig);
        s[k][j] = d * gate;
      }
      if (a.z) store_raw<GT, kV>((GT*)b.dz + row * a.D + c, pack_as<GT, kV>(dz));
      if (a.post_weight) {
        float pw[kV];
        load_vec(a.post_weight + c, pw);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          sums.add(0, k, j, s[k][j], p[k][j]);
          sums.add(1, k, j, s[k][j], 1.f);
          s[k][j] *= pw[j];
          m.x = fmaf(s[k][j], p[k][j], m.x);
          m.y += s[k][j];
        }
      }
    }
    if (a.post_weight) {
      m = g.sum(m);
      m.x *= a.inv_d;
      m.y = a.layer ? m.y * a.inv_d : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j) s[k][j] = ry * fmaf(-p[k][j], m.x, s[k][j] - m.y);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (g.column(k) < a.D)
        store_raw<GT, kV>((GT*)b.dy + row * a.D + g.column(k), pack_as<GT, kV>(s[k]));
  }
  // the groups' sums in group order (one group: the threads' own)
  float* dst[kSums] = {b.d_post_weight, b.d_post_bias, b.d_scale, b.d_weight, b.d_bias};
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    if (!dst[i]) continue;
    float* to = partial + ((long long)blockIdx.x * kSums + i) * a.D;
    if (g.count == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (g.column(k) + j < a.D) to[g.column(k) + j] = sums.get(i, k, j);
    } else {  // K = 1
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kV; ++j) shared[j * blockDim.x + threadIdx.x] = sums.get(i, 0, j);
      __syncthreads();
      for (int e = threadIdx.x; e < tpr * kV; e += blockDim.x) {
        const int j = e / tpr, lane = e % tpr;
        float t = 0.f;
        for (int q = 0; q < g.count; ++q) t += shared[j * blockDim.x + q * tpr + lane];
        if (lane * kV + j < a.D) to[lane * kV + j] = t;
      }
    }
  }
}

// Sums the blocks' partials in block order: 32 columns of one sum a block.
__global__ void __launch_bounds__(1024)
norm_bwd_sum_kernel(NormBwdArgs b, const float* partial, int blocks) {
  after_previous();
  __shared__ float part[32][33];
  float* dst[kSums] = {b.d_post_weight, b.d_post_bias, b.d_scale, b.d_weight, b.d_bias};
  float* to = dst[0];
#pragma unroll
  for (int i = 1; i < kSums; ++i)
    if (i == (int)blockIdx.y) to = dst[i];
  if (!to) return;
  const int D = b.f.D, c = blockIdx.x * 32 + threadIdx.x;
  float t = 0.f;
  if (c < D)
    for (int k = threadIdx.y; k < blocks; k += 32)
      t += partial[((long long)k * kSums + blockIdx.y) * D + c];
  part[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    for (int k = 1; k < 32; ++k) t += part[k][threadIdx.x];
    to[c] = t;
  }
}

// Blocks of the first launch: as many as the GPU holds at once.
int bwd_blocks(int rows, int D) {
  const Shape s = bwd_shape(D);
  const long long need = ((long long)rows + s.groups - 1) / s.groups;
  const int hold = 152 * (s.tpr * s.groups <= kThreads ? 2 : 1);
  return (int)(need < hold ? need : hold);
}

template <typename T, typename RT, typename GT, typename GRT>
cudaError_t run_bwd(const NormBwdArgs& b, float* partial, cudaStream_t stream) {
  const Shape s = bwd_shape(b.f.D);
  const int threads = s.tpr * s.groups, blocks = bwd_blocks(b.f.rows, b.f.D);
  int smem = s.groups * kRedFloats * 4;
  if (s.groups > 1 && smem < threads * kV * 4) smem = threads * kV * 4;
  if (s.k > 1) smem += kSums * s.k * kV * threads * 4;
  auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
    cudaError_t e = allow_shared(kernel, smem, done);
    if (e != cudaSuccess) return e;
    kernel<<<blocks, threads, smem, stream>>>(b, partial, s.tpr);
    return cudaGetLastError();
  };
  if (blocks > 0) {
    static std::atomic<uint64_t> done1{0}, done2{0};
    const cudaError_t e = s.k == 1 ? go(norm_bwd_kernel<T, RT, GT, GRT, 1>, done1)
                                   : go(norm_bwd_kernel<T, RT, GT, GRT, 2>, done2);
    if (e != cudaSuccess) return e;
  }
  if (!b.d_post_weight && !b.d_post_bias && !b.d_scale && !b.d_weight && !b.d_bias)
    return cudaSuccess;
  return launch_after(norm_bwd_sum_kernel, dim3((b.f.D + 31) / 32, kSums), dim3(32, 32), 0, stream,
                      b, (const float*)partial, blocks);
}

}  // namespace

size_t norm_bwd_workspace(int rows, int D) {
  return (size_t)bwd_blocks(rows, D) * kSums * D * 4;
}

cudaError_t launch_norm_bwd(const NormBwdArgs& b, void* workspace, cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  float* p = static_cast<float*>(workspace);
  if (b.f.fp32_io) return run_bwd<float, float, float, float>(b, p, stream);
  if (b.f.fp32_res)
    return b.f.fp32_out ? run_bwd<bf16, float, float, float>(b, p, stream)
                        : run_bwd<bf16, float, bf16, float>(b, p, stream);
  return b.f.fp32_out ? run_bwd<bf16, bf16, float, float>(b, p, stream)
                      : run_bwd<bf16, bf16, bf16, bf16>(b, p, stream);
}

}  // namespace gla
