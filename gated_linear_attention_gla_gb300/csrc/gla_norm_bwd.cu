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
// What takes the time: the latency of three exchanges a row, which 16 warps an SM do not hide (issue slots
// 54 % used, DRAM 41 %).  8192 x 2048, layer norm with biases, gate and scale 74 us, 3.6 TB/s; RMS 55 us, 4.9.
#include <type_traits>

#include "gla_norm.cuh"

namespace gla {
namespace {

using namespace norm;

constexpr int kSums = 4;  // A, B, d_weight, d_bias
// Rows of a group at a time: two, or one with two vectors a thread (whose sums lie in shared memory)
// and of the kernel for layer norm and biases, which holds 24 registers more and has four sums a
// row for one exchange (8192 x 2048, layer norm with biases: 93 us two at a time, 78 us one).
constexpr int rows_of(int kind) { return kind == kRms ? 2 : 1; }

// The sums of a thread's columns over the rows.
template <int K> struct Sums {
  Vec v[K == 1 ? kSums : 1];
  f32x2* s;  // K = 2: pair (i, k, j) at ((i K + k) kV / 2 + j) threads + thread
  __device__ void init(void* shared) {
    s = (f32x2*)shared + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      if constexpr (K == 1) {
        v[i] = vec_of(0.f);
      } else {
        for (int e = 0; e < K * kV / 2; ++e) s[(i * K * kV / 2 + e) * blockDim.x] = both(0.f);
      }
    }
  }
  __device__ __forceinline__ void add(int i, int k, int j, f32x2 x, f32x2 y) {
    if constexpr (K == 1) {
      v[i].v[j] = fma2(x, y, v[i].v[j]);
    } else {
      f32x2& t = s[((i * K + k) * kV / 2 + j) * blockDim.x];
      t = fma2(x, y, t);
    }
  }
  __device__ __forceinline__ f32x2 get(int i, int k, int j) const {
    if constexpr (K == 1) return v[i].v[j];
    else return s[((i * K + k) * kV / 2 + j) * blockDim.x];
  }
};

// R: rows at a time; KIND: kRms (without biases), or kEither of the norms with what biases there are
template <typename T, typename RT, typename GT, typename GRT, int K, int R, int KIND>
__global__ void __launch_bounds__(512, 1)
norm_bwd_kernel(NormBwdArgs b, float* partial, int tpr, int stages) {
  start_next();
  extern __shared__ __align__(16) unsigned char shared[];
  constexpr bool RMS = KIND == kRms, BIAS = !RMS;
  const NormArgs& a = b.f;
  const Group g(tpr, (float*)shared);
  // pieces of a row: res, ds, y, z, du
  constexpr int kDs = kPieces<RT>, kY = 2 * kDs, kZ = kY + kPieces<T>, kDu = kZ + kPieces<T>;
  Ring<K> ring(shared + g.count * kRedFloats * 4, R, kDu + kPieces<T>, stages);
  Sums<K> sums;
  sums.init(shared + g.count * kRedFloats * 4);  // (K = 2, which has no ring)
  Param<K> post, post_b, scale, weight;
  post.init(g, a.D, a.post_weight, 1.f);
  if (BIAS) post_b.init(g, a.D, a.post_bias, 0.f);
  scale.init(g, a.D, a.scale, 1.f);
  weight.init(g, a.D, a.weight, 1.f);
  const long long hop = (long long)gridDim.x * g.count * R;
  auto fetch = [&](long long row, int slot) {
    if constexpr (K == 1) {
      const int c = g.column(0);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool on = row + i < a.rows && c < a.D;
        const long long r = on ? row + i : 0;
        const int to = on ? c : 0;
        const long long at = r * a.D + to;
        ring.copy_or_0(slot, i, 0, (const RT*)a.res + at, on);
        if (b.d_res_out) ring.copy_or_0(slot, i, kDs, (const RT*)b.d_res_out + at, on);
        if (a.y) ring.copy_or_0(slot, i, kY, (const T*)a.y + r * a.y_stride + to, on);
        if (a.z) ring.copy_or_0(slot, i, kZ, (const T*)a.z + r * a.z_stride + to, on);
        if (b.d_out) ring.copy_or_0(slot, i, kDu, (const T*)b.d_out + at, on);
      }
      cp_commit();
    }
  };
  long long row = ((long long)blockIdx.x * g.count + g.index) * R;
  for (int i = 0; i < stages - 1; ++i) fetch(row + i * hop, i);
  for (; row < a.rows; row += hop, ring.next()) {
    fetch(row + (stages - 1) * hop, ring.ahead());
    ring.wait();
    // whether the thread has channels of row i
    const int rows = R == 1 || row + 1 >= a.rows ? 1 : 2;
    auto has = [&](int i, int k) { return g.column(k) < a.D && i < rows; };
    auto there = [&](int i, int k) { return K == 1 || has(i, k); };  // to be read
    // (columns and rows that do not exist are zeros, without branches between the rows;
    // of two vectors a thread those are skipped, whose parameters are not held)
    auto skip = [&](int k) { return K > 1 && g.column(k) >= a.D; };
    auto at = [&](int i, int k) { return (row + i) * a.D + g.column(k); };
    auto z_of = [&](int i, int k) {
      return there(i, k) ? ring.read(i, kZ, (const T*)a.z + (row + i) * a.z_stride + g.column(k))
                       : vec_of(0.f);
    };
    auto du_of = [&](int i, int k) {
      return there(i, k) ? ring.read(i, kDu, (const T*)b.d_out + at(i, k)) : vec_of(0.f);
    };
    auto ds_of = [&](int i, int k) {
      return b.d_res_out && there(i, k) ? ring.read(i, kDs, (const RT*)b.d_res_out + at(i, k))
                                      : vec_of(0.f);
    };
    Vec s[R][K], p[R][K];
    float ry[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      ry[i] = 1.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        s[i][k] = there(i, k) ? ring.read(i, 0, (const RT*)a.res + at(i, k)) : vec_of(0.f);
        p[i][k] = a.y && there(i, k)
                      ? ring.read(i, kY, (const T*)a.y + (row + i) * a.y_stride + g.column(k))
                      : vec_of(0.f);
      }
    }
    if (a.post_weight) {
      normalise<K, R, KIND>(g, a, p, ry, rows);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          GLA_PAIRS p[i][k].v[j] = mul2(p[i][k].v[j], both(ry[i]));
    }
    // q = p post_weight + post_bias, formed twice (again below) rather than held
    auto affine = [&](int i, int k) {
      const Vec w = post.at(g.column(k)), o = BIAS ? post_b.at(g.column(k)) : w;
      Vec q;
#pragma unroll
      GLA_PAIRS q.v[j] = BIAS ? fma2(p[i][k].v[j], w.v[j], o.v[j]) : mul2(p[i][k].v[j], w.v[j]);
      return q;
    };
    // s becomes d = dL/ds
    if (b.d_out) {
      if (a.y) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            if (skip(k)) continue;
            const Vec q = affine(i, k);
            Vec w = scale.at(g.column(k));
            if (a.z) {
              const Vec z = z_of(i, k);
#pragma unroll
              GLA_PAIRS w.v[j] = mul2(w.v[j], mul2(z.v[j], sigmoid2(z.v[j])));
            }
#pragma unroll
            GLA_PAIRS s[i][k].v[j] = fma2(w.v[j], q.v[j], s[i][k].v[j]);
          }
        }
      }
      float r[R], m[2 * R];
      if constexpr (RMS) {
        // mean(dn n) = r mean(dn s): its sum goes with that of the squares
#pragma unroll
        for (int i = 0; i < R; ++i) {
          f32x2 q = both(0.f), mx = both(0.f);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            if (skip(k)) continue;
            const Vec d = du_of(i, k), w = weight.at(g.column(k));
#pragma unroll
            GLA_PAIRS {
              q = fma2(s[i][k].v[j], s[i][k].v[j], q);
              mx = fma2(mul2(d.v[j], w.v[j]), s[i][k].v[j], mx);
            }
          }
          m[2 * i] = q.x + q.y;
          m[2 * i + 1] = mx.x + mx.y;
        }
        g.sum(m);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          r[i] = i < rows ? rsqrtf(fmaf(m[2 * i], a.inv_d, a.eps)) : 0.f;
          const f32x2 mx = both(-m[2 * i + 1] * r[i] * a.inv_d);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            if (skip(k)) continue;
            const Vec d = du_of(i, k), e = ds_of(i, k), w = weight.at(g.column(k));
#pragma unroll
            GLA_PAIRS {
              const f32x2 n = mul2(s[i][k].v[j], both(r[i]));
              sums.add(2, k, j, d.v[j], n);
              s[i][k].v[j] = fma2(both(r[i]), fma2(n, mx, mul2(d.v[j], w.v[j])), e.v[j]);
            }
          }
        }
      } else {
        // the same beside the sums of layer norm, whose mean comes out of both afterwards: mean(dn n) =
        // r (mean(dn s) - mean(s) mean(dn)), with normalise's second exchange where it has one
        static_assert(R == 1, "four sums at a time");
        float v[4] = {};
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (skip(k)) continue;
          const Vec d = du_of(0, k), w = weight.at(g.column(k));
          f32x2 t[4] = {};
#pragma unroll
          GLA_PAIRS {
            const f32x2 x = s[0][k].v[j], dn = mul2(d.v[j], w.v[j]);
            t[0] = add2(t[0], x);
            t[1] = fma2(x, x, t[1]);
            t[2] = add2(t[2], dn);
            t[3] = fma2(dn, x, t[3]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += t[e].x + t[e].y;
        }
        g.sum(v);
        const float mean = a.layer ? v[0] * a.inv_d : 0.f;
        float var = fmaf(-mean, mean, v[1] * a.inv_d), mx1 = fmaf(-mean, v[2], v[3]);
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (g.column(k) < a.D)
#pragma unroll
            GLA_PAIRS s[0][k].v[j] = add2(s[0][k].v[j], both(-mean));
        if (far_mean(mean, var)) {
          float c[2] = {};
#pragma unroll
          for (int k = 0; k < K; ++k) {
            if (skip(k)) continue;
            const Vec d = du_of(0, k), w = weight.at(g.column(k));
            f32x2 t[2] = {};
#pragma unroll
            GLA_PAIRS {
              t[0] = fma2(s[0][k].v[j], s[0][k].v[j], t[0]);
              t[1] = fma2(mul2(d.v[j], w.v[j]), s[0][k].v[j], t[1]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) c[e] += t[e].x + t[e].y;
          }
          g.sum(c);
          var = c[0] * a.inv_d;
          mx1 = c[1];
        }
        r[0] = rsqrtf(var + a.eps);
        const f32x2 mx = both(-mx1 * r[0] * a.inv_d);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (skip(k)) continue;
          // (columns that do not exist stay zeros: they are in the sums of the norm of y)
          const f32x2 my = both(a.layer && g.column(k) < a.D ? -v[2] * a.inv_d : 0.f);
          const Vec d = du_of(0, k), e = ds_of(0, k), w = weight.at(g.column(k));
#pragma unroll
          GLA_PAIRS {
            const f32x2 n = mul2(s[0][k].v[j], both(r[0]));
            sums.add(2, k, j, d.v[j], n);
            sums.add(3, k, j, d.v[j], both(1.f));
            s[0][k].v[j] = fma2(both(r[0]), fma2(n, mx, fma2(d.v[j], w.v[j], my)), e.v[j]);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) s[i][k] = ds_of(i, k);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (has(i, k)) store_vec((GRT*)b.d_res + at(i, k), s[i][k]);
    if (!a.y) continue;
    // s becomes dp, then dy
    constexpr int kMeans = RMS ? 1 : 2;
    float m[kMeans * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      f32x2 mx = both(0.f), my = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (skip(k)) continue;
        const int c = g.column(k);
        const Vec w = scale.at(c);
        if (a.z) {
          const Vec z = z_of(i, k);
          Vec q = affine(i, k);
#pragma unroll
          GLA_PAIRS {
            const f32x2 sig = sigmoid2(z.v[j]), gate = mul2(z.v[j], sig);
            // silu' = sig + gate (1 - sig)
            const f32x2 slope = fma2(gate, fma2(sig, both(-1.f), both(1.f)), sig);
            q.v[j] = mul2(q.v[j], mul2(mul2(s[i][k].v[j], w.v[j]), slope));  // dz
            s[i][k].v[j] = mul2(s[i][k].v[j], gate);
          }
          if (has(i, k)) store_vec((GT*)b.dz + at(i, k), q);
        }
#pragma unroll
        GLA_PAIRS {
          sums.add(0, k, j, s[i][k].v[j], p[i][k].v[j]);
          if (BIAS) sums.add(1, k, j, s[i][k].v[j], both(1.f));
          s[i][k].v[j] = mul2(s[i][k].v[j], w.v[j]);
        }
        if (a.post_weight) {
          const Vec pw = post.at(c);
#pragma unroll
          GLA_PAIRS {
            s[i][k].v[j] = mul2(s[i][k].v[j], pw.v[j]);
            mx = fma2(s[i][k].v[j], p[i][k].v[j], mx);
            my = add2(my, s[i][k].v[j]);
          }
        }
      }
      m[kMeans * i] = mx.x + mx.y;
      if (!RMS) m[kMeans * i + kMeans - 1] = my.x + my.y;
    }
    if (a.post_weight) {
      g.sum(m);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const f32x2 mx = both(-m[kMeans * i] * a.inv_d);
        const f32x2 my = both(a.layer ? -m[kMeans * i + kMeans - 1] * a.inv_d : 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          GLA_PAIRS s[i][k].v[j] =
              mul2(both(ry[i]),
                   fma2(p[i][k].v[j], mx, RMS ? s[i][k].v[j] : add2(s[i][k].v[j], my)));
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (has(i, k)) store_vec((GT*)b.dy + at(i, k), s[i][k]);
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
        GLA_PAIRS if (g.column(k) < a.D)
          *reinterpret_cast<float2*>(to + g.column(k) + 2 * j) = sums.get(i, k, j);
    } else {  // K = 1; the ring is free
      float* all = (float*)(shared + g.count * kRedFloats * 4);
      __syncthreads();
#pragma unroll
      GLA_PAIRS {
        const f32x2 t = sums.get(i, 0, j);
        all[2 * j * blockDim.x + threadIdx.x] = t.x;
        all[(2 * j + 1) * blockDim.x + threadIdx.x] = t.y;
      }
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

// Blocks of the first launch: as many as the GPU holds at once (and no more than rows).
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
  const int kind = bias || b.f.layer ? kEither : kRms;
  const int pieces = rows_of(kind) * (2 * kPieces<RT> + 3 * kPieces<T>);
  const int other = s.groups * kRedFloats * 4;
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
    auto of = [&](auto k) {
      constexpr int KIND = decltype(k)::value;
      static std::atomic<uint64_t> d0{0}, d1{0};
      return s.k == 1 ? go(norm_bwd_kernel<T, RT, GT, GRT, 1, rows_of(KIND), KIND>, d0)
                      : go(norm_bwd_kernel<T, RT, GT, GRT, 2, 1, KIND>, d1);
    };
    const cudaError_t e = kind == kRms ? of(std::integral_constant<int, kRms>())
                                       : of(std::integral_constant<int, kEither>());
    if (e != cudaSuccess) return e;
  }
  if (!b.d_post_weight && !b.d_post_bias && !b.d_scale && !b.d_weight && !b.d_bias)
    return cudaSuccess;
  return launch_after(norm_bwd_sum_kernel, dim3((b.f.D + 31) / 32, 2), dim3(32, 32), 0, stream, b,
                      (const float*)partial, blocks, (int)(kind != kRms));
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
