// gla_scan.cuh -- what the forward and backward scan kernels share.
#pragma once

#include "gla_ssm.cuh"

namespace gla {

// Prompts are cut into chunks of `chunk` tokens.  Sequence s owns the chunk slots
// from cu[s] / chunk + s on, which leaves room for ceil(length / chunk) of them
// for any lengths, so that a block finds its chunk without a table.
struct Chunk {
  long long t0, t1;  // rows
  int s;             // sequence
  bool ok, last;     // there is such a chunk; it is its sequence's last
};

__device__ __forceinline__ long long first_slot(const ScanArgs& p, int s, long long chunk) {
  const long long lo = p.cu_seqlens ? __ldg(p.cu_seqlens + s) : (long long)s * p.T;
  return lo / chunk + s;
}
__host__ __device__ inline long long slots_of(int B, long long rows, long long chunk) {
  return rows / chunk + B;
}
__device__ __forceinline__ long long rows_of(const ScanArgs& p) {
  return p.cu_seqlens ? (long long)p.T : (long long)p.B * p.T;
}

__device__ __forceinline__ Chunk chunk_of_slot(const ScanArgs& p, long long slot,
                                               long long chunk) {
  int lo = 0, hi = p.B - 1;  // the last s with first_slot(s) <= slot
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_slot(p, mid, chunk) <= slot) lo = mid;
    else hi = mid - 1;
  }
  long long a, b;
  seq_rows(p.cu_seqlens, lo, p.T, &a, &b);
  const long long c = slot - first_slot(p, lo, chunk);
  Chunk k;
  k.s = lo;
  k.ok = bounds_ok(a, b, rows_of(p)) && c >= 0 && a + c * chunk < b;
  k.t0 = a + c * chunk;
  k.t1 = min(k.t0 + chunk, b);
  k.last = k.t1 == b;
  return k;
}

// Sequence s's rows [*lo, *hi); false (and reported) for malformed offsets.
__device__ __forceinline__ bool seq_ok(const ScanArgs& p, int s, bool report, long long* lo,
                                       long long* hi) {
  seq_rows(p.cu_seqlens, s, p.T, lo, hi);
  const long long rows = rows_of(p);
  const bool ok = bounds_ok(*lo, *hi, rows) &&
                  (!p.cu_seqlens ||
                   (__ldg(p.cu_seqlens) == 0 && __ldg(p.cu_seqlens + p.B) == rows));
  if (!ok && report) atomicOr(p.status, kDevBadSeqlens);
  return ok;
}

// One recurrence over a sequence's chunks for four states of a channel: with
// `x` = log2(e) a, v[c] what chunk c adds and sum[c] its step sizes' sum,
// v[c] becomes the state in front of chunk c (from the last chunk on when
// `back`), starting from `run`, which ends as the state behind them all.
// Chunk c of the sequence is slot f + c; `per` float4s and D sums a slot.
__device__ __forceinline__ void scan_chunks(float4* v, const float* sum, float4 x, long long f,
                                            long long n, long long per, long long in, int D,
                                            int ch, bool back, float4* run) {
  constexpr int U = 16;
  for (long long c0 = 0; c0 < n; c0 += U) {
    float4 y[U];
    float w[U];
    long long at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long c = min(c0 + u, n - 1);
      at[u] = f + (back ? n - 1 - c : c);
      y[u] = v[at[u] * per + in];
      w[u] = sum[at[u] * D + ch];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u < n) {
        v[at[u] * per + in] = *run;
        run->x = fmaf(ex2(x.x * w[u]), run->x, y[u].x);
        run->y = fmaf(ex2(x.y * w[u]), run->y, y[u].y);
        run->z = fmaf(ex2(x.z * w[u]), run->z, y[u].z);
        run->w = fmaf(ex2(x.w * w[u]), run->w, y[u].w);
      }
    }
  }
}

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
