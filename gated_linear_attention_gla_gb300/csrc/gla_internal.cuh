// gla_internal.cuh -- declarations shared by the translation units of libgla.so.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

namespace gla {

// Bits of the per-GPU device status word (see gla_status_sync in gla.h).
enum : unsigned {
  kDevBadSeqlens = 1u << 0,  // a cu_seqlens entry was out of order or out of range
  kDevTimeout = 1u << 1,     // a bounded mbarrier wait gave up
  kDevLayout = 1u << 2,      // a kernel's shared-memory window was not 1024-byte aligned
  // (kDevBadSeqlens also flags a decode slot index outside the state pool, and a
  // page table's entry that names no page it could)
};

// Log-decays below -kGateClamp are raised to it before in-chunk cumulative
// sums, so that differences of sums stay finite (exp(-30) ~ 9.4e-14).
constexpr float kGateClamp = 30.0f;

struct ChunkArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  float scale;
  const float* init_state;
  void* out;
  float* final_state;
  const int32_t* cu_seqlens;
  int B, H, T, dk, dv, chunk;
  bool fp32_io;      // q, k, v (and out) fp32
  bool fp32_out;     // out fp32 with bf16 q, k, v
  bool vector_gate;
  bool out_reversed;  // token t of a sequence of len tokens stored at row len - 1 - t
                      // (tensor-core kernels only; the backward's reversed runs)
  // per-head tensor-core kernel only (the backward's dg terms): when dot_out is
  // set, dot_out[row, h] += dot_sign * sum_j out[row, h, j] * dot_rows[row, h, j]
  // (fp32 output values; dot_rows bf16 with the output's layout)
  const void* dot_rows;
  float* dot_out;
  float dot_sign;
  unsigned* status;   // device status word
};

struct DecodeArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  float scale;
  float* state;           // [N, H, dk, dv], or a pool of num_slots pages when slots is set
  const int32_t* slots;   // device [N]: the pool page of sequence n (-1: skip it), or null
  int num_slots;
  unsigned* status;       // device status word (slot out of range)
  void* out;
  // the mixer steps after the readout (each null = skipped): self-augmentation
  // weights [H, dk], head RMSNorm weights [H, dv] and eps, output gate [N, H, dv]
  const float* aug;
  const float* norm_w;
  float eps;
  const void* z;
  int N, H, dk, dv;
  bool fp32_io;
  bool fp32_out;
  bool vector_gate;
};

struct EpilogueArgs {
  void* out;              // [rows, H, dv], updated in place
  const void* q;          // [rows, H, dk] (with aug)
  const void* k;
  const void* v;          // [rows, H, dv] (with aug)
  const float* aug;       // [H, dk] or null
  const float* norm_w;    // [H, dv] or null
  float eps;
  const void* z;          // [rows, H, dv] or null
  long long rows;
  int H, dk, dv;
  bool fp32_io;           // q, k, v, z fp32 (else bf16)
  bool fp32_out;          // out fp32 (else bf16)
};

struct ChunkBwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  float scale;
  const float* init_state;  // [B, H, dk, dv] or null
  const void* d_out;        // [rows, H, dv]
  const float* d_final;     // [B, H, dk, dv] or null
  void* dq;
  void* dk;
  void* dv;
  float* dg;                // g's shape, or null
  float* d_init;            // [B, H, dk, dv] or null
  const int32_t* cu_seqlens;
  int B, H, T;
  int dk_size, dv_size;
  bool fp32_io;
  bool fp32_out;
  bool vector_gate;
  bool skip_dv;             // the CUDA-core kernels leave dv to another path
  unsigned* status;
};

// The short causal convolution (gla_conv_*): x [rows, D] with x_stride elements
// between rows, weight [D, W], states [B, W - 1, D] in x's dtype.
struct ConvArgs {
  const void* x;
  long long x_stride;
  const float* weight;
  const float* bias;        // [D] or null
  const void* init_state;   // or null
  void* out;                // [rows, D]
  void* final_state;        // or null; may be init_state
  const int32_t* cu_seqlens;
  int B, T, D, W;
  bool silu, fp32_io, fp32_out;
  unsigned* status;
};

struct ConvBwdArgs {
  const void* x;
  long long x_stride;
  const float* weight;
  const float* bias;
  const void* init_state;
  const void* d_out;           // [rows, D]
  const float* d_final_state;  // [B, W - 1, D] fp32 or null
  void* dx;                    // [rows, D]
  float* d_weight;             // [D, W]
  float* d_bias;               // [D] or null
  float* d_init_state;         // [B, W - 1, D] fp32 or null
  const int32_t* cu_seqlens;
  int B, T, D, W;
  bool silu, fp32_io, fp32_out;
  unsigned* status;
};

struct ConvStepArgs {
  const void* x;
  long long x_stride;
  const float* weight;
  const float* bias;
  void* state;              // [N, W - 1, D], or a pool of num_slots pages
  int num_slots;
  const int32_t* slots;     // pages read, or null
  const int32_t* out_slots; // pages written, or null: those read
  void* out;
  int N, D, W;
  bool silu, fp32_io, fp32_out;
  unsigned* status;
};

// The selective scan (gla_scan_*): u, dt, z [rows, D], b, c [rows, NS], each
// with its own row stride; a [D, NS]; states [B, D, NS] fp32.
struct ScanArgs {
  const void *u, *dt, *b, *c, *z;  // z may be null
  long long u_stride, dt_stride, b_stride, c_stride, z_stride;
  const float* a;
  const float* skip;     // [D] or null
  const float* dt_bias;  // [D] or null
  const float* init_state;
  void* out;
  float* final_state;
  const int32_t* cu_seqlens;
  int B, T, D, NS;
  bool softplus, fp32_io, fp32_out;
  unsigned* status;
};

struct ScanBwdArgs {
  ScanArgs f;                  // the forward's inputs (out and final_state unused)
  const void* d_out;           // [rows, D]
  const float* d_final_state;  // [B, D, NS] or null
  void *du, *ddt, *db, *dc, *dz;  // dz null without z
  float *da, *dskip, *ddt_bias;   // dskip, ddt_bias may be null
  float* d_init_state;            // or null
};

struct ScanStepArgs {
  const void *u, *dt, *b, *c, *z;
  long long u_stride, dt_stride, b_stride, c_stride, z_stride;
  const float* a;
  const float* skip;
  const float* dt_bias;
  float* state;
  int num_slots;
  const int32_t* slots;
  const int32_t* out_slots;
  void* out;
  int N, D, NS;
  bool softplus, fp32_io, fp32_out;
  unsigned* status;
};

// The norms, the gate and the residual sum between two blocks (gla_block_norm_*):
// y, z [rows, D] with row strides, res [rows, D]; the parameters [D] fp32.
struct NormArgs {
  const void* res;
  const void* y;             // or null: s = res
  const void* z;             // or null
  long long y_stride, z_stride;
  const float* post_weight;  // or null: no norm of y
  const float* post_bias;    // or null
  const float* scale;        // or null
  const float* weight;
  const float* bias;         // or null
  float eps, inv_d;          // inv_d = 1 / D
  void* res_out;             // or null; may be res
  void* out;                 // or null: no norm of s
  int rows, D;
  bool layer, fp32_io, fp32_res, fp32_out;
};

struct NormBwdArgs {
  NormArgs f;                // the forward's inputs (res_out, out, bias unused)
  const void* d_out;         // [rows, D] or null: zero
  const void* d_res_out;     // [rows, D] or null: zero
  void *d_res, *dy, *dz;     // dy, dz null without y, z
  // [D] each, or null: not computed
  float *d_post_weight, *d_post_bias, *d_scale, *d_weight, *d_bias;
};

// The gated linear recurrence (gla_recur_*): x, f, i, z [rows, D] with row
// strides; states [B, D] fp32.
struct RecurArgs {
  const void *x, *f, *i, *z;  // i and z may be null
  long long x_stride, f_stride, i_stride, z_stride;
  const float* decay;         // [D] or null
  const float* init_state;    // or null
  void* out;
  float* final_state;
  const int32_t* cu_seqlens;
  int B, T, D;
  bool unit, fp32_io, fp32_out;
  unsigned* status;
  uint64_t wait_ns;           // limit of a wait
};

struct RecurBwdArgs {
  RecurArgs f;                 // the forward's inputs (out and final_state unused)
  const void* d_out;           // [rows, D]
  const float* d_final_state;  // [B, D] or null
  void *dx, *df, *di, *dz;     // di, dz null without i, z
  float* d_decay;              // or null without decay
  float* d_init_state;         // or null
};

struct RecurStepArgs {
  const void *x, *f, *i, *z;
  long long x_stride, f_stride, i_stride, z_stride;
  const float* decay;
  float* state;
  int num_slots;
  const int32_t* slots;
  const int32_t* out_slots;
  void* out;
  int N, D;
  bool unit, fp32_io, fp32_out;
  unsigned* status;
};

// The gated feed-forward projections (gla_glu_*), bf16: x [rows, D] with
// x_stride elements between rows, weights [F, D].
struct GluArgs {
  const void* x;
  long long x_stride;
  const void* w_gate;
  const void* w_up;
  void* out;             // [rows, F]
  int rows, D, F;
  bool fp32_out;
  unsigned* status;
};

struct GluBwdArgs {
  GluArgs f;             // the forward's inputs (out unused)
  const void* d_out;     // [rows, F]
  void *dx, *dw_gate, *dw_up;
};

// One pool of state pages: page i at base + i * page_bytes.
struct PagePool {
  void* base;
  long long page_bytes;
};
constexpr int kMaxPools = 64;  // pools of one copy launch
struct PagePools {
  char* base[kMaxPools];
  long long bytes[kMaxPools];
  int first[kMaxPools];  // index of the pool's first slice
  int count;
};
constexpr int kPageNew = -2;       // gla.h's GLA_PAGE_NEW
constexpr int kMaxPages = 524288;  // pages of a pool (the copy plan keeps three bits a page)

// Wall-time limit of the hand-off waits of the tensor-core prefill, the projections and the gated
// recurrence, read at each launch (process-wide; set by gla_set_wait_limit_ns, default 2 s).  Their
// teardown drains keep limits of their own.
constexpr uint64_t kDefaultWaitLimitNs = 2000000000ull;
uint64_t handoff_wait_limit_ns();

// Kernel launchers (one per translation unit).  They assume validated arguments
// and a non-empty problem, and return the launch error.
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_epilogue(const EpilogueArgs& a, cudaStream_t stream);
cudaError_t launch_chunk_simt(const ChunkArgs& a, cudaStream_t stream);
bool chunk_tc_supported(const ChunkArgs& a);
cudaError_t launch_chunk_tc(const ChunkArgs& a, cudaStream_t stream);
bool chunk_tc_vec_supported(const ChunkArgs& a);
// with `mix`, the mixer's steps after the readout run inside the kernel (the
// fields other than aug, norm_w, eps and z are ignored)
cudaError_t launch_chunk_tc_vec(const ChunkArgs& a, cudaStream_t stream,
                                const EpilogueArgs* mix = nullptr);
// the chunked backward, one launcher per (gate, I/O dtype)
cudaError_t launch_chunk_bwd_head_bf16(const ChunkBwdArgs& a, cudaStream_t stream);
cudaError_t launch_chunk_bwd_head_f32(const ChunkBwdArgs& a, cudaStream_t stream);
cudaError_t launch_chunk_bwd_chan_bf16(const ChunkBwdArgs& a, cudaStream_t stream);
cudaError_t launch_chunk_bwd_chan_f32(const ChunkBwdArgs& a, cudaStream_t stream);
// the backward on the tensor cores, bf16, with chunk_bwd_tc_workspace(B, H,
// rows, dk, dv, vector_gate) bytes of workspace: per-head gate (d_k, d_v in
// {64, 128}), every gradient from three prefill runs; per-key-channel gate
// (d_k = d_v = 128), dv from one run of the per-key-channel prefill (dq, dk on
// the CUDA cores)
bool chunk_bwd_tc_supported(int dk, int dv, bool fp32_io, bool vector_gate);
size_t chunk_bwd_tc_workspace(int B, int H, long long rows, int dk, int dv, bool vector_gate);
cudaError_t launch_chunk_bwd_tc(const ChunkBwdArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_chunk_bwd_tc_vec_dv(const ChunkBwdArgs& a, void* workspace,
                                       cudaStream_t stream);
cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t stream);
size_t conv_bwd_workspace(long long rows, int D, int W);
cudaError_t launch_conv_bwd(const ConvBwdArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t stream);
// workspace bytes of a scan (0: none) and the scan itself
size_t scan_fwd_workspace(int B, long long rows, int D, int NS, bool packed);
cudaError_t launch_scan_fwd(const ScanArgs& a, void* workspace, cudaStream_t stream);
size_t scan_bwd_workspace(int B, long long rows, int D, int NS);
cudaError_t launch_scan_bwd(const ScanBwdArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t stream);
constexpr int kNormMaxD = 8192;
cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream);
size_t norm_bwd_workspace(int rows, int D);
cudaError_t launch_norm_bwd(const NormBwdArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_recur_fwd(const RecurArgs& a, cudaStream_t stream);
size_t recur_bwd_workspace(int B, long long rows, int D, bool packed);
cudaError_t launch_recur_bwd(const RecurBwdArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_recur_step(const RecurStepArgs& a, cudaStream_t stream);
cudaError_t launch_glu_fwd(const GluArgs& a, cudaStream_t stream);
// A tile of dw sums over all rows, 64 of them in 0.34 us: 2^26 take 0.36 s, a fifth of the default limit of
// the wait for them (2^29 would end as a wait that ran out).
constexpr int kGluBwdMaxRows = 1 << 26;
size_t glu_bwd_workspace(int rows, int D, int F);
cudaError_t launch_glu_bwd(const GluBwdArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_pages_copy(const PagePool* pools, int count, int S, const int32_t* src,
                              const int32_t* dst, int32_t* plan, int n, unsigned* status,
                              cudaStream_t stream);
cudaError_t launch_pages_fork(const PagePool* pools, int count, int S, const int32_t* used,
                              int32_t* used_out, const int32_t* parents, int32_t* children,
                              int n, unsigned* status, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagePool* pools, int count, int S, const int32_t* used,
                                 int32_t* used_out, const int32_t* slots, int32_t* slots_out,
                                 int n, int32_t* forward, unsigned* status, cudaStream_t stream);
cudaError_t launch_pages_free(int S, const int32_t* used, int32_t* used_out,
                              const int32_t* slots, int n, unsigned* status,
                              cudaStream_t stream);
// what the entry points share (gla_api.cu): the current GPU's status word, a
// CUDA result remembered for gla_last_error_string as a status, range checks
unsigned* device_status_word(cudaError_t* err);
int cuda_result(cudaError_t e);
// the fixed device workspace of gla_chunk_bwd_fixed_workspace (a static array;
// its address, or null with *err set)
constexpr size_t kBwdFixedWorkspaceBytes = 384ull << 20;
void* bwd_fixed_workspace(cudaError_t* err);

// ---------------------------------------------------------------------------
// Small device helpers shared by the kernels.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Lets a kernel use `bytes` of dynamic shared memory (above the 48 KB every kernel
// may).  The attribute belongs to the current device: `done` (one per kernel)
// remembers, by device, where it has been set.
template <typename K>
inline cudaError_t allow_shared(K kernel, int bytes, std::atomic<uint64_t>& done) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A launch that may overlap its own start with the end of the launch before it on
// the stream (programmatic dependent launch).  The kernel calls after_previous()
// before it touches memory, so it sees everything the launch before has
// written; what a chain of such launches wrote is complete when its last one is.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, int smem,
                                cudaStream_t stream, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = stream;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next launch of such a chain start (its blocks then wait for this
// launch's end): for kernels of one block or one wave, which leave SMs empty at
// their end.
__device__ __forceinline__ void start_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Sequence bounds for sequence s: dense batches own rows [s*T, s*T+T); packed
// batches read cu_seqlens.  Returns false (and flags the status word) for a
// malformed entry.
__device__ __forceinline__ bool seq_bounds(const int32_t* cu, int s, int B, int T,
                                           long long* start, int* len, unsigned* status) {
  if (cu == nullptr) {
    *start = (long long)s * T;
    *len = T;
    return true;
  }
  const int a = __ldg(cu + s), b = __ldg(cu + s + 1);
  const int first = __ldg(cu), last = __ldg(cu + B);
  if (first != 0 || last != T || a < 0 || b < a || b > T) {
    if (status) atomicOr(status, kDevBadSeqlens);
    return false;
  }
  *start = a;
  *len = b - a;
  return true;
}

}  // namespace gla
