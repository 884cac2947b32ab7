// gla_norm_bwd.cu -- the gradient of the norms, the gate and the residual sum between two
// blocks, from the forward's inputs alone.  With n = norm(s), p = norm(y) without
// their weights, q = p post_weight + post_bias, r the factors 1 / sqrt(mean + eps):
//     d_weight = sum du n,  d_bias = sum du
//     d = ds + r_s (dn - mean(dn) - n mean(dn n)),   dn = du weight     (mean(dn): layer norm)
//     d_res = d,  d_scale = sum d q silu(z),  dz = d scale q silu'(z)
//     dq = d scale silu(z),  d_post_weight = sum dq p,  d_post_bias = sum dq
//     dy = r_y (dp - mean(dp) - p mean(dp p)),       dp = dq post_weight
// One pass: a group of threads owns a row as in the forward (whose values it
// computes again) and walks over rows.  Of the sums over rows four suffice, A = sum d silu(z) p,
// B = sum d silu(z), d_weight and d_bias: d_post_weight = scale A, d_post_bias = scale B,
// d_scale = post_weight A + post_bias B.  They stay with the thread that owns the
// column (in registers; in shared memory where a thread holds two vectors, whose
// sums would not fit), are summed over a block's groups and written as one partial a
// block, which a second launch sums in block order.  No atomics: the same inputs
// give the same bits.
// Bound: HBM.
#include "gla_norm.cuh"

namespace gla {
namespace {

using namespace norm;

constexpr int kSums = 4;  // A, B, d_weight, d_bias

// The sums of a thread's columns over the rows.
template <int K> struct Sums {
  float v[K == 1 ? kSums : 1][K == 1 ? kV : 1];
  float* s;  // K = 2: element (i, k, j) at ((i K + k) kV + j) threads + thread
  __device__ void init(float* shared) {
    s = shared + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          if constexpr (K == 1) v[i][j] = 0.f;
          else s[((i * K + k) * kV + j) * blockDim.x] = 0.f;
        }
  }
  __device__ __forceinline__ void add(int i, int k, int j, float x, float y) {
    if constexpr (K == 1) {
      v[i][j] = fmaf(x, y, v[i][j]);
    } else {
      float& t = s[((i * K + k) * kV + j) * blockDim.x];
      t = fmaf(x, y, t);
    }
  }
  __device__ __forceinline__ float get(int i, int k, int j) const {
    if constexpr (K == 1) return v[i][j];
    else return s[((i * K + k) * kV + j) * blockDim.x];
  }
};

// BIAS: layer norm's biases (post_bias, d_post_bias, d_bias)
template <typename T, typename RT, typename GT, typename GRT, int K, bool BIAS>
__global__ void __launch_bounds__(512, 1)
norm_bwd_kernel(NormBwdArgs b, float* partial, int tpr, int stages) {
  start_next();
  extern __shared__ __align__(16) unsigned char shared[];
  const NormArgs& a = b.f;
  const Group g(tpr, (float*)shared);
  // pieces of a row: res, ds, y, z, du
  constexpr int kDs = kPieces<RT>, kY = 2 * kDs, kZ = kY + kPieces<T>, kDu = kZ + kPieces<T>;
  Ring<K> ring(shared + g.count * kRedFloats * 4, kDu + kPieces<T>, stages);
  Sums<K> sums;
  sums.init((float*)(shared + g.count * kRedFloats * 4));  // (K = 2, which has no ring)
  Param<K> post, post_b, scale, weight;
  post.init(g, a.D, a.post_weight, 1.f);
  if (BIAS) post_b.init(g, a.D, a.post_bias, 0.f);
  scale.init(g, a.D, a.scale, 1.f);
  weight.init(g, a.D, a.weight, 1.f);
  const long long hop = (long long)gridDim.x * g.count;
  auto fetch = [&](long long row, int slot) {
    if constexpr (K == 1) {
      const int c = g.column(0);
      if (row < a.rows && c < a.D) {
        ring.copy(slot, 0, (const RT*)a.res + row * a.D + c);
        if (b.d_res_out) ring.copy(slot, kDs, (const RT*)b.d_res_out + row * a.D + c);
        if (a.y) ring.copy(slot, kY, (const T*)a.y + row * a.y_stride + c);
        if (a.z) ring.copy(slot, kZ, (const T*)a.z + row * a.z_stride + c);
        if (b.d_out) ring.copy(slot, kDu, (const T*)b.d_out + row * a.D + c);
      }
      cp_commit();
    }
  };
  long long row = (long long)blockIdx.x * g.count + g.index;
  for (int i = 0; i < stages - 1; ++i) fetch(row + i * hop, i);
  for (; row < a.rows; row += hop, ring.next()) {
    fetch(row + (stages - 1) * hop, ring.ahead());
    ring.wait();
    const long long at = row * a.D;
    const T* zr = (const T*)a.z + row * a.z_stride;
    float s[K][kV], p[K][kV];
    float ry = 1.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      fill(s[k], 0.f);
      fill(p[k], 0.f);
      if (g.column(k) < a.D) {
        ring.read(0, (const RT*)a.res + at + g.column(k), s[k]);
        if (a.y) ring.read(kY, (const T*)a.y + row * a.y_stride + g.column(k), p[k]);
      }
    }
    if (a.post_weight) {
      ry = normalise<K>(g, a, p);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j) p[k][j] *= ry;
    }
    // q = p post_weight + post_bias, formed twice (again below) rather than held
    auto affine = [&](int k, float (&q)[kV]) {
      float w[kV], o[kV];
      post.at(g.column(k), w);
      if (BIAS) post_b.at(g.column(k), o);
#pragma unroll
      for (int j = 0; j < kV; ++j) q[j] = BIAS ? fmaf(p[k][j], w[j], o[j]) : p[k][j] * w[j];
    };
    // s becomes d = dL/ds
    if (b.d_out) {
      if (a.y) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (g.column(k) >= a.D) continue;
          float q[kV], w[kV];
          affine(k, q);
          scale.at(g.column(k), w);
          if (a.z) {
            float z[kV];
            ring.read(kZ, zr + g.column(k), z);
#pragma unroll
            for (int j = 0; j < kV; ++j) w[j] *= silu(z[j]);
          }
#pragma unroll
          for (int j = 0; j < kV; ++j) s[k][j] = fmaf(w[j], q[j], s[k][j]);
        }
      }
      const float r = normalise<K>(g, a, s);
      float2 m = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (g.column(k) >= a.D) continue;
        float d[kV], w[kV];
        ring.read(kDu, (const T*)b.d_out + at + g.column(k), d);
        weight.at(g.column(k), w);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const float n = s[k][j] * r;
          s[k][j] = n;
          sums.add(2, k, j, d[j], n);
          if (BIAS) sums.add(3, k, j, d[j], 1.f);
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
        ring.read(kDu, (const T*)b.d_out + at + g.column(k), d);
        fill(e, 0.f);
        if (b.d_res_out) ring.read(kDs, (const RT*)b.d_res_out + at + g.column(k), e);
        weight.at(g.column(k), w);
#pragma unroll
        for (int j = 0; j < kV; ++j)
          s[k][j] = fmaf(r, fmaf(-s[k][j], m.x, fmaf(d[j], w[j], -m.y)), e[j]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        fill(s[k], 0.f);
        if (b.d_res_out && g.column(k) < a.D) 
          ring.read(kDs, (const RT*)b.d_res_out + at + g.column(k), s[k]);
      }
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
      float w[kV];
      scale.at(c, w);
      if (a.z) {
        float z[kV], q[kV];
        affine(k, q);
        ring.read(kZ, zr + c, z);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const float sig = sigmoid(z[j]), gate = z[j] * sig, d = s[k][j] * gate;
          q[j] *= s[k][j] * w[j] * fmaf(gate, 1.f - sig, sig);  // dz
          s[k][j] = d;
        }
        store_raw<GT, kV>((GT*)b.dz + row * a.D + c, pack_as<GT, kV>(q));
      }
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        sums.add(0, k, j, s[k][j], p[k][j]);
        if (BIAS) sums.add(1, k, j, s[k][j], 1.f);
        s[k][j] *= w[j];
      }
      if (a.post_weight) {
        float pw[kV];
        post.at(c, pw);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
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
  cp_wait<0>();
  // the groups' sums in group order (one group: the threads' own)
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    if (!BIAS && i % 2 == 1) continue;
    float* to = partial + ((long long)blockIdx.x * kSums + i) * a.D;
    if (g.count == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (g.column(k) + j < a.D) to[g.column(k) + j] = sums.get(i, k, j);
    } else {  // K = 1; the ring is free
      float* all = (float*)(shared + g.count * kRedFloats * 4);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kV; ++j) all[j * blockDim.x + threadIdx.x] = sums.get(i, 0, j);
      __syncthreads();
      for (int e = threadIdx.x; e < tpr * kV; e += blockDim.x) {
        const int j = e / tpr, lane = e % tpr;
        float t = 0.f;
        for (int q = 0; q < g.count; ++q) t += all[j * blockDim.x + q * tpr + lane];
        if (lane * kV + j < a.D) to[lane * kV + j] = t;
      }
    }
  }
}

// Sums the blocks' partials in block order, 32 columns of a pair of sums a block: A and B
// (blockIdx.y 0), or d_weight and d_bias.
__global__ void __launch_bounds__(1024)
norm_bwd_sum_kernel(NormBwdArgs b, const float* partial, int blocks, int bias) {
  after_previous();
  __shared__ float2 part[32][33];
  const int D = b.f.D, c = blockIdx.x * 32 + threadIdx.x;
  float2 t = make_float2(0.f, 0.f);
  if (c < D)
    for (int k = threadIdx.y; k < blocks; k += 32) {
      const float* from = partial + ((long long)k * kSums + 2 * blockIdx.y) * D + c;
      t.x += from[0];
      if (bias) t.y += from[D];
    }
  part[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y != 0 || c >= D) return;
  for (int k = 1; k < 32; ++k) t = add2(t, part[k][threadIdx.x]);
  if (blockIdx.y == 1) {
    if (b.d_weight) b.d_weight[c] = t.x;
    if (b.d_bias) b.d_bias[c] = t.y;
    return;
  }
  const float sc = b.f.scale ? b.f.scale[c] : 1.f;
  const float w = b.f.post_weight ? b.f.post_weight[c] : 1.f;
  const float o = b.f.post_bias ? b.f.post_bias[c] : 0.f;
  if (b.d_post_weight) b.d_post_weight[c] = sc * t.x;
  if (b.d_post_bias) b.d_post_bias[c] = sc * t.y;
  if (b.d_scale) b.d_scale[c] = fmaf(w, t.x, o * t.y);
}

// Blocks of the first launch: as many as the GPU holds at once.
int bwd_blocks(int rows, int D) {
  const Shape s = shape_of(D);
  const long long need = ((long long)rows + s.groups - 1) / s.groups;
  const int hold = 152 * (s.tpr * s.groups <= 256 ? 2 : 1);
  return (int)(need < hold ? need : hold);
}

template <typename T, typename RT, typename GT, typename GRT>
cudaError_t run_bwd(const NormBwdArgs& b, float* partial, cudaStream_t stream) {
  const Shape s = shape_of(b.f.D);
  const int threads = s.tpr * s.groups, blocks = bwd_blocks(b.f.rows, b.f.D);
  const bool bias = b.f.post_bias || b.d_bias;
  const int pieces = 2 * kPieces<RT> + 3 * kPieces<T>, other = s.groups * kRedFloats * 4;
  const int stages = s.k == 1 ? ring_stages(pieces, threads, other, threads <= 256 ? 2 : 1) : 1;
  int room = s.k == 1 ? stages * pieces * 16 * threads : kSums * s.k * kV * threads * 4;
  if (room < threads * kV * 4) room = threads * kV * 4;  // the groups' sums at the end
  auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
    const cudaError_t e = allow_shared(kernel, 227 * 1024, done);
    if (e != cudaSuccess) return e;
    kernel<<<blocks, threads, other + room, stream>>>(b, partial, s.tpr, stages);
    return cudaGetLastError();
  };
  if (blocks > 0) {
    static std::atomic<uint64_t> d0{0}, d1{0}, d2{0}, d3{0};
    const cudaError_t e =
        s.k == 1 ? (bias ? go(norm_bwd_kernel<T, RT, GT, GRT, 1, true>, d0)
                         : go(norm_bwd_kernel<T, RT, GT, GRT, 1, false>, d1))
                 : (bias ? go(norm_bwd_kernel<T, RT, GT, GRT, 2, true>, d2)
                         : go(norm_bwd_kernel<T, RT, GT, GRT, 2, false>, d3));
    if (e != cudaSuccess) return e;
  }
  if (!b.d_post_weight && !b.d_post_bias && !b.d_scale && !b.d_weight && !b.d_bias)
    return cudaSuccess;
  return launch_after(norm_bwd_sum_kernel, dim3((b.f.D + 31) / 32, 2), dim3(32, 32), 0, stream, b,
                      (const float*)partial, blocks, (int)bias);
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
