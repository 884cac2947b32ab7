// gla_pages.cu -- the pages of state pools: copying, forking, compacting and
// freeing, without the host in between.
//
// A sequence's recurrent state is one page of fixed size in every pool (one
// pool per layer and kind of state), all under the same page number.  A table
// `used` (int32 per page, 0 = free) says which pages are taken.  Each operator
// is a plan -- one block that reads the tables and decides, in page order, so
// that the answer never depends on scheduling -- and, where pages move, a copy
// over all pools at HBM bandwidth that reads the plan.
//
// 256 pages of 1 MB moved by a compaction: 85 us, 93 % of copy bandwidth; 256 forks in
// eight pools (142 MB read, 142 MB written): 48 us, 87 %.  A few small pages: 7 us, the
// latency of two launches and of the plan's passes over the tables.
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kPlan = 1024;          // threads of the planning block
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;         // 16-byte vectors in flight per thread
constexpr long long kSlice = (long long)kCopyThreads * kCopyVecs * 16;  // bytes a block copies

// Exclusive prefix sum of a flag over the block, and the block's total.
__device__ __forceinline__ int block_rank(bool flag, int* total) {
  __shared__ int warp_sum[kPlan / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();  // the previous call's sums have been read
  if (lane == 0) warp_sum[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
  const int v = warp_sum[lane];
#pragma unroll
  for (int w = 0; w < kPlan / 32; ++w) {
    const int x = __shfl_sync(0xffffffffu, v, w);
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + __popc(m & ((1u << lane) - 1u));
}

// children[i] = the page taken for parents[i]: the free pages in ascending
// order, one for each entry that can be served, in entry order.
__global__ void __launch_bounds__(kPlan)
fork_plan_kernel(const int32_t* used, int32_t* used_out, int S, const int32_t* parents,
                 int32_t* children, int n, unsigned* status) {
  start_next();
  const int tid = threadIdx.x;
  auto wants = [&](int i) {
    const int p = parents[i];
    return p == kPageNew || (p >= 0 && p < S && used[p] != 0);
  };
  // how many entries ask for a page
  int asked = 0;
  bool bad = false;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + tid;
    const bool w = i < n && wants(i);
    bad |= i < n && !w && parents[i] != -1;
    asked += __syncthreads_count(w);
  }
  // the first `asked` free pages, listed in children[0 ..)
  int found = 0;
  for (int base = 0; base < S && found < asked; base += kPlan) {
    const int p = base + tid;
    const bool free_page = p < S && used[p] == 0;
    int total;
    const int rank = found + block_rank(free_page, &total);
    if (free_page && rank < asked) children[rank] = p;
    found += total;
  }
  __syncthreads();
  // each entry's page, from the end: entry i takes listed page rank(i) <= i
  int left = asked;
  for (int base = n > 0 ? (n - 1) / kPlan * kPlan : -1; base >= 0; base -= kPlan) {
    const int i = base + tid;
    const bool w = i < n && wants(i);
    int total;
    const int rank = block_rank(w, &total);
    left -= total;
    const int at = left + rank;
    const int page = w && at < found ? children[at] : -1;
    bad |= w && page < 0;  // no page is left
    __syncthreads();
    if (i < n) children[i] = page;
  }
  // the table last: it may be updated in place
  __syncthreads();
  if (used_out != used)
    for (int p = tid; p < S; p += kPlan) used_out[p] = used[p];
  __syncthreads();
  for (int i = tid; i < n; i += kPlan)
    if (children[i] >= 0) used_out[children[i]] = 1;
  if (bad) atomicOr(status, kDevBadSeqlens);
}

// forward[p] = the page that page p's contents go to: with L pages used, the
// k-th used page at or behind L (ascending) goes to the k-th free page in
// front of L, every other used page stays; -1 for a free page.
__global__ void __launch_bounds__(kPlan)
compact_plan_kernel(const int32_t* used, int32_t* used_out, int S, const int32_t* slots,
                    int32_t* slots_out, int n, int32_t* forward, unsigned* status) {
  start_next();
  const int tid = threadIdx.x;
  int L = 0;
  for (int base = 0; base < S; base += kPlan)
    L += __syncthreads_count(base + tid < S && used[base + tid] != 0);
  // the free pages in front of L, listed in forward[L ..): there are as many
  // as used pages behind, at most S - L
  int holes = 0;
  for (int base = 0; base < L; base += kPlan) {
    const int p = base + tid;
    const bool hole = p < L && used[p] == 0;
    int total;
    const int rank = holes + block_rank(hole, &total);
    if (hole) forward[L + rank] = p;
    if (p < L) forward[p] = hole ? -1 : p;
    holes += total;
  }
  __syncthreads();
  // the pages behind, from the end: page p takes listed hole rank(p) <= p - L
  int left = holes;
  for (int base = S > L ? (S - L - 1) / kPlan * kPlan : -1; base >= 0; base -= kPlan) {
    const int p = L + base + tid;
    const bool far = p < S && used[p] != 0;
    int total;
    const int rank = block_rank(far, &total);
    left -= total;
    const int to = far ? forward[L + left + rank] : -1;
    __syncthreads();
    if (p < S) forward[p] = to;
  }
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < n; i += kPlan) {
    const int s = slots[i];
    const bool ok = s >= 0 && s < S && used[s] != 0;
    bad |= !ok && s != -1;
    slots_out[i] = ok ? forward[s] : -1;
  }
  __syncthreads();  // the table last: it may be updated in place
  for (int p = tid; p < S; p += kPlan) used_out[p] = p < L ? 1 : 0;
  if (bad) atomicOr(status, kDevBadSeqlens);
}

// plan[i] = dst[i] where pair i can be copied beside all others: both pages in
// the pool, no other pair writes dst[i], and no other pair reads it.  Else -1.
__global__ void __launch_bounds__(kPlan)
copy_plan_kernel(const int32_t* src, const int32_t* dst, int n, int S, int32_t* plan,
                 unsigned* status) {
  start_next();
  extern __shared__ unsigned bits[];  // three maps of S bits: written, written twice, read
  const int words = (S + 31) / 32, tid = threadIdx.x;
  for (int i = tid; i < 3 * words; i += kPlan) bits[i] = 0u;
  __syncthreads();
  auto inside = [&](int s, int d) { return s >= 0 && s < S && d >= 0 && d < S; };
  for (int i = tid; i < n; i += kPlan) {
    const int s = src[i], d = dst[i];
    if (!inside(s, d)) continue;
    const unsigned bit = 1u << (d & 31);
    if (atomicOr(&bits[d >> 5], bit) & bit) atomicOr(&bits[words + (d >> 5)], bit);
    if (s != d) atomicOr(&bits[2 * words + (s >> 5)], 1u << (s & 31));
  }
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < n; i += kPlan) {
    const int s = src[i], d = dst[i];
    const bool skip = s == -1 || d == -1;
    bool ok = inside(s, d);
    if (ok) {
      const unsigned bit = 1u << (d & 31);
      ok = !(bits[words + (d >> 5)] & bit) && !(bits[2 * words + (d >> 5)] & bit);
    }
    bad |= !ok && !skip;
    plan[i] = ok ? d : -1;
  }
  if (bad) atomicOr(status, kDevBadSeqlens);
}

__global__ void __launch_bounds__(kPlan)
free_kernel(const int32_t* used, int32_t* used_out, int S, const int32_t* slots, int n,
            unsigned* status) {
  const int tid = threadIdx.x;
  if (used_out != used)
    for (int p = tid; p < S; p += kPlan) used_out[p] = used[p];
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < n; i += kPlan) {
    const int s = slots[i];
    if (s >= 0 && s < S) bad |= atomicExch(&used_out[s], 0) == 0;  // freed before, or twice
    else bad |= s != -1;
  }
  if (bad) atomicOr(status, kDevBadSeqlens);
}

// Block (x, y): slice x of the pools' pages laid end to end, pairs y, y +
// gridDim.y, ...; src null: pair i is page i.  A block's loads are all in
// flight before its first store.
__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(const PagePools pools, const int32_t* src, const int32_t* dst, int n) {
  after_previous();
  int q = 0;
  while (q + 1 < pools.count && (int)blockIdx.x >= pools.first[q + 1]) ++q;
  const long long off = ((long long)blockIdx.x - pools.first[q]) * kSlice;
  const long long page = pools.bytes[q];
  const int vecs = (int)(min(kSlice, page - off) / 16);
  char* base = pools.base[q] + off;
  for (int i = blockIdx.y; i < n; i += gridDim.y) {
    const int to = dst[i];
    const int from = src ? src[i] : i;
    if (to < 0 || to == from) continue;
    uint4* d = reinterpret_cast<uint4*>(base + to * page);
    uint4 v[kCopyVecs];
    if (from == kPageNew) {
#pragma unroll
      for (int k = 0; k < kCopyVecs; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4* s = reinterpret_cast<const uint4*>(base + from * page);
#pragma unroll
      for (int k = 0; k < kCopyVecs; ++k) {
        const int at = k * kCopyThreads + threadIdx.x;
        if (at < vecs) v[k] = __ldcs(s + at);
      }
    }
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k) {
      const int at = k * kCopyThreads + threadIdx.x;
      if (at < vecs) __stcs(d + at, v[k]);
    }
  }
}

cudaError_t copy_pages(const PagePool* list, int count, const int32_t* src, const int32_t* dst,
                       int n, cudaStream_t stream) {
  for (int first = 0; first < count && n > 0; first += kMaxPools) {
    PagePools p{};
    p.count = count - first < kMaxPools ? count - first : kMaxPools;
    int slices = 0;
    for (int i = 0; i < p.count; ++i) {
      p.base[i] = static_cast<char*>(list[first + i].base);
      p.bytes[i] = list[first + i].page_bytes;
      p.first[i] = slices;
      slices += (int)((p.bytes[i] + kSlice - 1) / kSlice);
    }
    if (slices > 0) {
      // (pairs beyond 256 in turn: a compaction's list has every page, most of
      // which stay)
      const cudaError_t e =
          launch_after(copy_pages_kernel, dim3((unsigned)slices, (unsigned)(n < 256 ? n : 256)),
                       dim3(kCopyThreads), 0, stream, p, src, dst, n);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_pages_copy(const PagePool* pools, int count, int S, const int32_t* src,
                              const int32_t* dst, int32_t* plan, int n, unsigned* status,
                              cudaStream_t stream) {
  // the limit for the largest pool, once: set to a call's own size, it would take from
  // another thread's call between that one's setting and its launch
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(copy_plan_kernel, 3 * (kMaxPages / 32) * 4, done);
  if (e != cudaSuccess) return e;
  copy_plan_kernel<<<1, kPlan, 3 * ((S + 31) / 32) * 4, stream>>>(src, dst, n, S, plan, status);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : copy_pages(pools, count, src, plan, n, stream);
}

cudaError_t launch_pages_fork(const PagePool* pools, int count, int S, const int32_t* used,
                              int32_t* used_out, const int32_t* parents, int32_t* children,
                              int n, unsigned* status, cudaStream_t stream) {
  fork_plan_kernel<<<1, kPlan, 0, stream>>>(used, used_out, S, parents, children, n, status);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : copy_pages(pools, count, parents, children, n, stream);
}

cudaError_t launch_pages_compact(const PagePool* pools, int count, int S, const int32_t* used,
                                 int32_t* used_out, const int32_t* slots, int32_t* slots_out,
                                 int n, int32_t* forward, unsigned* status,
                                 cudaStream_t stream) {
  compact_plan_kernel<<<1, kPlan, 0, stream>>>(used, used_out, S, slots, slots_out, n, forward,
                                               status);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : copy_pages(pools, count, nullptr, forward, S, stream);
}

cudaError_t launch_pages_free(int S, const int32_t* used, int32_t* used_out,
                              const int32_t* slots, int n, unsigned* status,
                              cudaStream_t stream) {
  free_kernel<<<1, kPlan, 0, stream>>>(used, used_out, S, slots, n, status);
  return cudaGetLastError();
}

}  // namespace gla
