/*
 * gla.h -- C ABI of libgla.so: gated linear attention (GLA) on one NVIDIA
 * GB300 (sm_103a).
 *
 * The method (the "i14 Laplace 3B on AWS Trainium2" blog page, section
 * "i14 and the Laplace 3B architecture", paragraph "GLA mixer"): every head
 * keeps a dk x dv matrix state S that decays and absorbs one rank-1
 * key/value write per token, and the query reads the state after the write:
 *
 *     S_t = diag(exp g_t) S_{t-1} + k_t^T v_t
 *     o_t = scale * q_t S_t
 *
 * g_t is a log-decay, either one value per (token, head) -- the page's
 * "Simple GLA" with a per-head decay -- or one value per (token, head, key
 * channel), where row i of S decays by exp(g_t[i]).
 *
 * Entry points:
 *   gla_chunk_fwd    prefill: the chunked form of the same page's section
 *                    "Challenge 1" (Figure 3) -- per chunk a causal Q K^T
 *                    weighted by the decays, times V, plus the carried-in
 *                    state's share, then one state step with the chunk's
 *                    total decay; emits the final state.
 *   gla_decode_step  one token for each of N concurrent sequences, each with a
 *                    fixed-size state page updated in place (section
 *                    "Inference optimization on Trainium2": one fixed page per
 *                    sequence); gla_decode_step_slots takes the pages from a
 *                    pool by slot index (for padded, graph-replayed batches).
 *   gla_mixer_epilogue, gla_chunk_fwd_mixer, gla_decode_step_mixer
 *                    the mixer's steps after the readout (self-augmentation,
 *                    head RMSNorm, SiLU output gate): over a finished output,
 *                    after a prefill in one call, fused into the decode step.
 *   gla_chunk_bwd    the gradient of the prefill (dq, dk, dv, dg and the
 *                    initial state's gradient) for training;
 *                    gla_chunk_bwd_workspace_size sizes its tensor-core path's
 *                    workspace, gla_chunk_bwd_fixed_workspace runs it on a
 *                    buffer of the library's own.
 *   gla_conv_fwd, gla_conv_bwd, gla_conv_step
 *                    the short causal convolution in front of a selective scan:
 *                    prompts, gradients, one token over a pool of states.
 *   gla_scan_fwd, gla_scan_bwd, gla_scan_step
 *                    the selective state space scan, whose decay differs for
 *                    every channel, state and token: likewise.
 *   gla_recur_fwd, gla_recur_bwd, gla_recur_step
 *                    a gated linear recurrence with one state per channel:
 *                    prompts, gradients, one token over a pool of states.
 *   gla_block_norm_fwd, gla_block_norm_bwd
 *                    between two blocks: norm, gate, residual sum, norm.
 *   gla_glu_fwd, gla_glu_bwd
 *                    the gated feed-forward projections and their product.
 *   gla_pages_copy, gla_pages_fork, gla_pages_compact, gla_pages_free
 *                    the pages of state pools, managed on the device.
 *   gla_status_sync, gla_status_string, gla_last_error_string, gla_version,
 *   gla_chunk_fwd_kernel, gla_set_wait_limit_ns
 *                    diagnostics.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates or frees device memory; it keeps one device status word
 *     per GPU and the fixed backward workspace (static __device__ variables)
 *     and no other state.
 *   - Calls are asynchronous on `stream` (0 = legacy default stream).  Host-side
 *     argument checks happen before anything is enqueued: a call that returns
 *     an error has launched nothing and written nothing.
 *   - Layouts are dense, row-major, token-major ("[B, T, H, d]": d fastest).
 *   - bf16 is IEEE-style bfloat16 (1-8-7); outputs are rounded to nearest even
 *     from fp32.  States are fp32 (the convolution's, which hold inputs, in the
 *     inputs' dtype).  Accumulation is fp32.
 *   - Errors detected on the device (a malformed cu_seqlens, an internal wait
 *     that ran out) set bits in the status word; the affected (sequence, head)
 *     writes nothing.  gla_status_sync() reports and clears them.
 *   - Thread safety: calls may come from any host thread; the device status
 *     word is shared by all streams of a GPU.
 */
#ifndef GLA_H_
#define GLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream; declared here so that this header
 * needs no CUDA header. */
typedef struct CUstream_st *gla_stream_t;

typedef enum gla_status {
    GLA_OK = 0,
    GLA_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad flags, bad cu_seqlens */
    GLA_ERR_UNSUPPORTED = 2,  /* valid but not implemented: head size, chunk size */
    GLA_ERR_MISALIGNED = 3,   /* a tensor pointer is not 16-byte aligned */
    GLA_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed */
    GLA_ERR_TIMEOUT = 5       /* a bounded on-device wait gave up (reported by gla_status_sync) */
} gla_status;

/* flags */
#define GLA_FLAG_FP32_IO (1u << 0)     /* q, k, v and out are fp32 (default bf16) */
#define GLA_FLAG_VECTOR_GATE (1u << 1) /* g has one value per key channel (default per head) */
#define GLA_FLAG_FP32_OUT (1u << 2)    /* out is fp32 while q, k, v stay bf16; the bf16 output of
                                          the same call is exactly this result rounded to
                                          nearest-even (same kernels, only the store differs) */
#define GLA_FLAG_SILU (1u << 3)        /* gla_conv_*: silu after the convolution */
#define GLA_FLAG_SOFTPLUS (1u << 4)    /* gla_scan_*: the step size is softplus(dt + dt_bias)
                                          (default dt + dt_bias) */
#define GLA_FLAG_UNIT_VARIANCE (1u << 5) /* gla_recur_*: the drive's factor is sqrt(1 - a^2)
                                          (default 1 - a) */
#define GLA_FLAG_LAYER_NORM (1u << 6)  /* gla_block_norm_*: norms subtract the mean (default RMS) */
#define GLA_FLAG_FP32_RESIDUAL (1u << 7) /* gla_block_norm_*: the residual rows are fp32 while the
                                          others stay bf16 */

/*
 * gla_chunk_fwd -- chunked prefill over a batch of sequences.
 *
 * Source: "i14 Laplace 3B" page, section "Challenge 1: Using native PyTorch
 * on Trainium for GLA" (chunked intra-chunk output, chunked state update,
 * Figure 3), with the recurrence of the "GLA mixer" paragraph.  Chunks start
 * at each sequence start; the last chunk of a sequence may be partial.  The
 * chunk size changes only the rounding, not the result.
 *
 * Arguments
 *   q, k        [B, T, H, dk] (dense) or [R, H, dk] (packed), bf16 or fp32
 *   v           [B, T, H, dv] or [R, H, dv], same dtype as q
 *   g           fp32 log-decay, [B, T, H] / [R, H], or with
 *               GLA_FLAG_VECTOR_GATE [B, T, H, dk] / [R, H, dk].  Values must be
 *               <= 0 or -inf; values below -30 act as -30 (exp(-30) ~ 1e-13).
 *   scale       readout scale (finite), usually dk^-0.5
 *   init_state  fp32 [B, H, dk, dv] state before the first token, or NULL (zeros)
 *   out         [B, T, H, dv] / [R, H, dv], same dtype as q (fp32 with
 *               GLA_FLAG_FP32_OUT); must not overlap any input
 *   final_state fp32 [B, H, dk, dv] state after the last token, or NULL (not
 *               written).  May alias init_state exactly (in-place update).
 *   cu_seqlens  NULL for a dense batch of B sequences of T tokens; otherwise a
 *               DEVICE int32 [B+1] array of packed sequence offsets with
 *               cu_seqlens[0] = 0, non-decreasing, cu_seqlens[B] = T = R (the
 *               number of packed token rows).  Checked on the device: a
 *               violation sets GLA_ERR_INVALID_ARG in the status word and the
 *               offending sequence writes nothing.
 *   B, H, T     batch (or number of packed sequences), heads, tokens per
 *               sequence (or packed rows).  B, H, T >= 0; with T = 0 (or empty
 *               sequences) final_state receives init_state (or zeros).
 *   dk, dv      head sizes: dk 64, 96 or 128; dv 64, 128 or 192
 *   chunk       tokens per chunk: 128 (tensor-core path for bf16 I/O: the
 *               per-head gate with every head size above -- dk = 64 and 96
 *               run zero-padded to 128 --, the per-key-channel gate with
 *               dk = dv = 128), or 16, 32, 64 (fp32 SIMT path); fp32 I/O and
 *               the other head sizes take the SIMT path
 *   stream      CUDA stream
 *   flags       GLA_FLAG_* bits; 0 = bf16 I/O, per-head gate
 *
 * Alignment: q, k, v, out, init_state, final_state must be 16-byte aligned; g
 * 4-byte aligned (16-byte with GLA_FLAG_VECTOR_GATE).
 */
gla_status gla_chunk_fwd(const void *q, const void *k, const void *v, const float *g,
                         float scale, const float *init_state, void *out,
                         float *final_state, const int32_t *cu_seqlens, int B, int H,
                         int T, int dk, int dv, int chunk, gla_stream_t stream,
                         unsigned flags);

/*
 * gla_decode_step -- one recurrent step for N concurrent sequences.
 *
 * Source: "i14 Laplace 3B" page, paragraph "GLA mixer" (the recurrence, one
 * token) and section "Inference optimization on Trainium2" (decode over many
 * concurrent sequences, one fixed state page per sequence).
 *
 * For every (n, h): S <- diag(exp g) S + k^T v (in place), o <- scale * q S.
 *
 * Arguments
 *   q, k         [N, H, dk], bf16 or fp32 (GLA_FLAG_FP32_IO)
 *   v            [N, H, dv], same dtype
 *   g            fp32 [N, H], or [N, H, dk] with GLA_FLAG_VECTOR_GATE; -inf allowed
 *   scale        readout scale
 *   state_inout  fp32 [N, H, dk, dv], read and overwritten in place
 *   out          [N, H, dv], same dtype as q (fp32 with GLA_FLAG_FP32_OUT)
 *   N, H         sequences and heads (>= 0; 0 does nothing)
 *   dk, dv       dk 64, 96 or 128; dv 64, 128 or 192
 * Alignment: every pointer 16-byte aligned except g (4-byte).
 */
gla_status gla_decode_step(const void *q, const void *k, const void *v, const float *g,
                           float scale, float *state_inout, void *out, int N, int H,
                           int dk, int dv, gla_stream_t stream, unsigned flags);

/*
 * gla_decode_step_slots -- the decode step with the states held in a pool of
 * pages, sequence n using page slots[n].
 *
 * Source: as gla_decode_step; the page's serving setup keeps one fixed state
 * page per sequence in a pool that the token mixer reads and writes (section
 * "Inference optimization on Trainium2").  Indexing the pool lets sequences
 * arrive and leave without moving state, and lets a batch be padded to a
 * fixed width (for CUDA-graph replay) with rows that do nothing.
 *
 * Arguments: as gla_decode_step, except
 *   state_pool   fp32 [num_slots, H, dk, dv]; page slots[n] is read and
 *                overwritten in place for sequence n
 *   num_slots    pages in the pool (>= 0)
 *   slots        DEVICE int32 [N]: the page of each row.  -1 marks a padding
 *                row: its state is not touched and its out row not written.
 *                The slots of one call must be distinct (two rows on one page
 *                race).  A slot >= num_slots is reported by gla_status_sync
 *                as GLA_ERR_INVALID_ARG and that row does nothing.
 * Returns GLA_ERR_INVALID_ARG for a null slots pointer; alignment as
 * gla_decode_step (slots 4-byte aligned).
 */
gla_status gla_decode_step_slots(const void *q, const void *k, const void *v, const float *g,
                                 float scale, float *state_pool, int num_slots,
                                 const int32_t *slots, void *out, int N, int H, int dk, int dv,
                                 gla_stream_t stream, unsigned flags);

/*
 * gla_mixer_epilogue -- the mixer's steps after the readout, in place over a
 * finished output (for instance the out of gla_chunk_fwd).
 *
 * Source: "i14 Laplace 3B" page, paragraph "GLA mixer": a self-augmentation
 * adds the value gated by the query dotted with a learned per-key-channel
 * rescaling of the key; the per-head outputs pass a head RMSNorm (one weight
 * per decay tier); the result is gated by SiLU of the gate stream.  Per token
 * and head, each step skipped when its pointer is null:
 *     o += sigmoid(sum_i q_i aug[h][i] k_i) * v
 *     o  = o / sqrt(mean_j o_j^2 + eps) * norm_w[h][j]
 *     o *= z / (1 + exp(-z))
 *
 * Arguments
 *   out          [rows, H, dv] bf16 (fp32 with GLA_FLAG_FP32_OUT), in place
 *   q, k         [rows, H, dk], v [rows, H, dv]: bf16 (fp32 with
 *                GLA_FLAG_FP32_IO); needed only with aug
 *   aug          fp32 [H, dk] or NULL
 *   norm_w       fp32 [H, dv] or NULL (a tier's heads carry equal rows)
 *   eps          >= 0, added to the mean square
 *   z            [rows, H, dv], q's dtype, or NULL
 *   rows, H      token rows and heads (>= 0); dk, dv as gla_chunk_fwd
 *   flags        GLA_FLAG_FP32_IO, GLA_FLAG_FP32_OUT only
 * Alignment: every pointer 16-byte aligned.  out must not overlap any input.
 */
gla_status gla_mixer_epilogue(void *out, const void *q, const void *k, const void *v,
                              const float *aug, const float *norm_w, float eps, const void *z,
                              int rows, int H, int dk, int dv, gla_stream_t stream,
                              unsigned flags);

/*
 * gla_chunk_fwd_mixer -- gla_chunk_fwd followed by the mixer's steps after the
 * readout (as gla_mixer_epilogue) on its output, in one call: the prefill, then
 * a second launch over `out` (a pass at ~70 % of HBM bandwidth).  Arguments:
 * those of gla_chunk_fwd, plus aug, norm_w, eps and z as for
 * gla_mixer_epilogue (z shaped like out, in q's dtype); each step is skipped
 * when its pointer is NULL.  Alignment: as gla_chunk_fwd, and aug, norm_w, z
 * 16-byte aligned.
 */
gla_status gla_chunk_fwd_mixer(const void *q, const void *k, const void *v, const float *g,
                               float scale, const float *init_state, void *out,
                               float *final_state, const int32_t *cu_seqlens, int B, int H,
                               int T, int dk, int dv, int chunk, const float *aug,
                               const float *norm_w, float eps, const void *z,
                               gla_stream_t stream, unsigned flags);

/*
 * gla_decode_step_mixer -- the decode step with the mixer's steps after the
 * readout fused into it (one CTA owns a head's whole output row).
 *
 * Arguments: as gla_decode_step_slots (slots NULL: state is [N, H, dk, dv]
 * and num_slots must be 0), plus aug, norm_w, eps and z as for
 * gla_mixer_epilogue (z [N, H, dv] in q's dtype).  Each step is skipped when
 * its pointer is NULL.
 */
gla_status gla_decode_step_mixer(const void *q, const void *k, const void *v, const float *g,
                                 float scale, float *state, int num_slots,
                                 const int32_t *slots, void *out, int N, int H, int dk, int dv,
                                 const float *aug, const float *norm_w, float eps,
                                 const void *z, gla_stream_t stream, unsigned flags);

/*
 * gla_chunk_bwd -- the gradient of gla_chunk_fwd (training), for a loss whose
 * gradients with respect to out and final_state are d_out and d_final_state.
 *
 * Source: "i14 Laplace 3B" page, section "Challenge 1" (the chunked layer is
 * trained; its backward pass runs over the chunks like the forward) with the
 * recurrence of the "GLA mixer" paragraph.  Reverse mode through
 * S_t = diag(exp g_t) S_{t-1} + k_t^T v_t, o_t = scale q_t S_t: with
 * Sbar_t = dL/dS_t = scale q_t^T do_t + diag(exp g_{t+1}) Sbar_{t+1},
 *     dq_t = scale S_t do_t^T      dk_t = Sbar_t v_t^T      dv_t = k_t Sbar_t
 *     dg_t[i] = exp(g_t[i]) sum_j S_{t-1}[i][j] Sbar_t[i][j]  (summed over i
 *               for the per-head gate)
 *     d_init = diag(exp g_0) Sbar_0
 * computed chunk by chunk (64 tokens) in fp32.  The gate is clamped at -30 as
 * in the forward; dg is the gradient with respect to the clamped gate.
 *
 * Arguments
 *   q, k, v, g, scale, init_state, cu_seqlens, B, H, T, dk, dv
 *                 exactly as passed to gla_chunk_fwd
 *   d_out         [B, T, H, dv] / [R, H, dv], q's dtype: dL/d out
 *   d_final_state fp32 [B, H, dk, dv] dL/d final_state, or NULL (zero)
 *   dq, dk_out    [.., H, dk]; dv_out [.., H, dv]: q's dtype, fp32 with
 *                 GLA_FLAG_FP32_OUT (the bf16 results are these rounded to
 *                 nearest-even)
 *   dg            fp32, g's shape, or NULL (not computed).  With the per-head
 *                 gate its terms are summed across CTAs with fp32 atomics, so
 *                 its last bits may vary from run to run.
 *   d_init_state  fp32 [B, H, dk, dv], or NULL (not written)
 *   workspace     device scratch owned by the caller, or NULL; with at least
 *                 gla_chunk_bwd_workspace_size(...) bytes (256-byte aligned),
 *                 bf16 I/O and dk, dv each 64 or 128 (the per-key-channel
 *                 gate: dk = dv = 128), the call uses the tensor cores:
 *                 the gradient of the recurrence is the same recurrence with
 *                 its operands exchanged -- dq is the prefill of (d_out, v, k),
 *                 dk and dv are prefills of (v, d_out, q) and (k, q, d_out) run
 *                 backwards in time.  Per-head gate: the tcgen05 prefill kernel
 *                 runs three times between a reversing pass and a tail pass
 *                 (dg's final-state term and suffix sums, d_init's factor);
 *                 each run stores its gradient straight into dq, dk_out or
 *                 dv_out, and the dq and dk runs add dg's per-token terms
 *                 with fp32 atomics.  Per-key-channel gate: dv is one reversed run of the
 *                 per-key-channel tcgen05 prefill (whose decay falls on the
 *                 state's rows, as dv's does); dq and dk, whose decays fall on
 *                 the value side, stay on the CUDA cores.  Tensor-core results
 *                 have the prefill's accuracy (bf16 operands, fp32
 *                 accumulation).  Otherwise (or with a smaller workspace) the
 *                 fp32 CUDA-core kernels run.
 *   flags         GLA_FLAG_FP32_IO, GLA_FLAG_VECTOR_GATE, GLA_FLAG_FP32_OUT
 * The outputs and the workspace must not overlap one another or any input.
 * Empty sequences write d_init_state = d_final_state (or zeros).
 * Alignment: as gla_chunk_fwd; every output 16-byte aligned.
 */
gla_status gla_chunk_bwd(const void *q, const void *k, const void *v, const float *g,
                         float scale, const float *init_state, const void *d_out,
                         const float *d_final_state, void *dq, void *dk_out, void *dv_out,
                         float *dg, float *d_init_state, const int32_t *cu_seqlens, int B,
                         int H, int T, int dk, int dv, void *workspace,
                         size_t workspace_bytes, gla_stream_t stream, unsigned flags);

/*
 * gla_chunk_bwd_fixed_workspace -- gla_chunk_bwd for callers that cannot
 * allocate device memory when they need the gradient (code running inside a
 * caching allocator's callbacks, real-time threads that must not take the
 * driver's allocation lock, embedders whose memory is reserved up front): the
 * tensor-core path takes its workspace from a fixed device buffer inside the
 * library, so the call allocates nothing (no cudaMalloc, no cudaFree, no
 * allocating library routine).  The pages have no counterpart of this entry
 * point; it is a deployment convenience.
 *
 * The buffer is a static device array of GLA_BWD_FIXED_WORKSPACE_BYTES
 * (384 MiB).  With CUDA's lazy module loading (CUDA_MODULE_LOADING=LAZY, the
 * default) it is placed on a GPU the first time this function needs it there;
 * with eager loading every process that loads libgla.so reserves it on every
 * GPU it uses, forward-only users included.  Once placed it stays until the
 * process exits.  The first call that needs it on a device looks up its
 * device address (cudaGetSymbolAddress) and caches it: make that first call
 * before capturing any stream into a CUDA graph.  If the buffer cannot be
 * placed (not enough free memory when the module loads), the call returns
 * GLA_ERR_CUDA with the runtime's reason in gla_last_error_string(), and the
 * runtime's last-error state is cleared so that later calls are not charged
 * with it.
 *
 * Sizes: a call whose workspace need (gla_chunk_bwd_workspace_size) exceeds
 * the buffer is rejected with GLA_ERR_UNSUPPORTED before anything is enqueued,
 * and gla_last_error_string() states the need and the limit (with d_k = d_v =
 * 128 and 16 heads the buffer covers about 20,000 tokens, e.g. ten sequences
 * of 2,048);
 * such a call can go to gla_chunk_bwd with workspace = NULL, which runs the
 * CUDA-core kernels and needs no workspace either.  Calls that the tensor-core
 * path does not cover (fp32 I/O, other head sizes) need no workspace and run
 * on the CUDA cores as with gla_chunk_bwd.
 *
 * Sharing: every call on a GPU uses the same buffer, and a call overwrites
 * what the previous one left there (each call writes every workspace byte it
 * reads, so nothing depends on earlier contents).  Calls that overlap in time
 * on the GPU race on it: issue them on one stream, or synchronise between them.
 * Arguments, results and errors otherwise as gla_chunk_bwd.
 */
#define GLA_BWD_FIXED_WORKSPACE_BYTES ((size_t)384 << 20)
gla_status gla_chunk_bwd_fixed_workspace(const void *q, const void *k, const void *v,
                                         const float *g, float scale, const float *init_state,
                                         const void *d_out, const float *d_final_state,
                                         void *dq, void *dk_out, void *dv_out, float *dg,
                                         float *d_init_state, const int32_t *cu_seqlens, int B,
                                         int H, int T, int dk, int dv, gla_stream_t stream,
                                         unsigned flags);

/*
 * gla_chunk_bwd_workspace_size -- bytes of device workspace with which
 * gla_chunk_bwd takes its tensor-core path for these sizes and flags, or 0 when
 * that path does not cover them (the call then runs on the CUDA cores and
 * needs no workspace).  `packed` != 0: T counts packed rows (cu_seqlens given).
 * Pure host function.
 */
size_t gla_chunk_bwd_workspace_size(int B, int H, int T, int dk, int dv, int packed,
                                    unsigned flags);

/*
 * gla_chunk_fwd_kernel -- which kernel gla_chunk_fwd runs for a non-empty call
 * with these head sizes, chunk size and flags: "tensor_core" (a tcgen05
 * kernel: per-head or per-key-channel gate), "cuda_core" (the fp32 CUDA-core
 * kernel), or NULL when the call would be rejected.  Pure host function:
 * launches nothing.
 */
const char *gla_chunk_fwd_kernel(int dk, int dv, int chunk, unsigned flags);

/*
 * The selective-scan layer.  Its parts that carry state: a short causal
 * convolution per channel, and a state space scan whose decay and drive depend
 * on the token.  (Projections before, between and after them are matrix
 * products.)  The pages the recurrence above comes from have no counterpart;
 * these entry points stand beside it for layers whose decay is one value per
 * (channel, state, token), which no matrix product over a chunk covers.
 *
 * Shared by the six entry points below
 *   - Tokens are rows: row b * T + t of a dense batch, or packed rows with
 *     cu_seqlens as for gla_chunk_fwd (a malformed cu_seqlens is reported by
 *     gla_status_sync as GLA_ERR_INVALID_ARG; the call's outputs are then
 *     unspecified, nothing outside them is written).
 *   - x, u, dt, z, b and c take the distance between rows in elements
 *     (x_stride, ...), so that they may be column slices of one projection's
 *     output.  Every other tensor is contiguous.
 *   - D, the channels, is a multiple of 8, at most 2^24.  Rows of x, u, dt, z
 *     start on 16 bytes (pointer and stride); b and c rows on an element.
 *   - Parameters (weight, bias, a, skip, dt_bias) and their gradients are fp32;
 *     weight, bias and a start on 16 bytes.
 *   - Gradients come in the inputs' dtype, or fp32 with GLA_FLAG_FP32_OUT; they
 *     are summed in a fixed order (the same inputs give the same bits).
 *   - Outputs and workspaces must not overlap one another or any input.
 */

/*
 * gla_conv_fwd -- p[t][d] = bias[d] + sum_j weight[d][W-1-j] x[t-j][d],
 * out = p, or p / (1 + exp(-p)) with GLA_FLAG_SILU.
 *
 *   x            [rows, D], bf16 or fp32 (GLA_FLAG_FP32_IO)
 *   weight       [D, W], W = 2, 3 or 4; bias [D] or NULL
 *   init_state   [B, W-1, D] in x's dtype: the W-1 rows before each sequence,
 *                oldest first, or NULL (zeros)
 *   out          [rows, D], x's dtype (fp32 with GLA_FLAG_FP32_OUT)
 *   final_state  [B, W-1, D] in x's dtype: the last W-1 rows (of init_state
 *                and x), or NULL.  May be init_state itself.
 */
gla_status gla_conv_fwd(const void *x, int64_t x_stride, const float *weight, const float *bias,
                        const void *init_state, void *out, void *final_state,
                        const int32_t *cu_seqlens, int B, int T, int D, int W,
                        gla_stream_t stream, unsigned flags);

/*
 * gla_conv_bwd -- the gradient of gla_conv_fwd.  d_out [rows, D] in x's dtype;
 * d_final_state and d_init_state [B, W-1, D] fp32, or NULL (zero; not
 * written); dx [rows, D]; d_weight [D, W]; d_bias [D] or NULL.  workspace:
 * gla_conv_bwd_workspace_size(...) bytes of device memory, 256-byte aligned.
 */
gla_status gla_conv_bwd(const void *x, int64_t x_stride, const float *weight, const float *bias,
                        const void *init_state, const void *d_out, const float *d_final_state,
                        void *dx, float *d_weight, float *d_bias, float *d_init_state,
                        const int32_t *cu_seqlens, int B, int T, int D, int W, void *workspace,
                        size_t workspace_bytes, gla_stream_t stream, unsigned flags);
size_t gla_conv_bwd_workspace_size(int B, int T, int D, int W, int packed);

/*
 * gla_conv_step -- one token for each of N sequences.  x, out [N, D];
 * state [N, W-1, D] in x's dtype, shifted by x in place; with slots (DEVICE
 * int32 [N]) a pool of num_slots pages, as for gla_decode_step_slots.
 * out_slots (DEVICE int32 [N], or NULL for slots): the page that receives row
 * n's new state; page slots[n] is then left as it was, and several rows may
 * read the same page (a fork during the step).  The pages written by one call
 * must be distinct, and none may be read by another row.  A row with -1 in
 * either table does nothing.
 */
gla_status gla_conv_step(const void *x, int64_t x_stride, const float *weight, const float *bias,
                         void *state, int num_slots, const int32_t *slots,
                         const int32_t *out_slots, void *out, int N, int D, int W,
                         gla_stream_t stream, unsigned flags);

/*
 * gla_scan_fwd -- for every sequence, channel d and state n = 0 .. N-1
 *     delta  = dt + dt_bias[d], or softplus of it with GLA_FLAG_SOFTPLUS
 *     h[t][d][n] = exp(delta a[d][n]) h[t-1][d][n] + delta u[t][d] b[t][n]
 *     out[t][d]  = (sum_n c[t][n] h[t][d][n] + skip[d] u[t][d]) z / (1 + exp(-z))
 *
 *   u, dt        [rows, D]; b, c [rows, N]: bf16, or fp32 with GLA_FLAG_FP32_IO
 *   a            [D, N], finite; N = 8, 16, 32 or 64 (16-byte aligned).  Either
 *                sign, as delta without GLA_FLAG_SOFTPLUS: decays may exceed 1.
 *                Where their product over a stretch of a sequence leaves fp32's
 *                range, what follows from it is infinite or NaN.
 *   skip, dt_bias  [D] or NULL (zero)
 *   z            [rows, D] or NULL (no gate); z_stride is then ignored
 *   init_state   fp32 [B, D, N] or NULL (zeros); final_state likewise or NULL
 *                (not written), may be init_state itself
 *   out          [rows, D], u's dtype (fp32 with GLA_FLAG_FP32_OUT)
 *   workspace    gla_scan_fwd_workspace_size(...) bytes (256-byte aligned; NULL
 *                where that is 0)
 */
gla_status gla_scan_fwd(const void *u, int64_t u_stride, const void *dt, int64_t dt_stride,
                        const float *a, const void *b, int64_t b_stride, const void *c,
                        int64_t c_stride, const float *skip, const void *z, int64_t z_stride,
                        const float *dt_bias, const float *init_state, void *out,
                        float *final_state, const int32_t *cu_seqlens, int B, int T, int D,
                        int N, void *workspace, size_t workspace_bytes, gla_stream_t stream,
                        unsigned flags);
size_t gla_scan_fwd_workspace_size(int B, int T, int D, int N, int packed);

/*
 * gla_scan_bwd -- the gradient of gla_scan_fwd.  d_out [rows, D] in u's dtype;
 * d_final_state, d_init_state fp32 [B, D, N] or NULL; du, ddt, dz [rows, D]
 * (dz NULL exactly without z); db, dc [rows, N]; da [D, N]; dskip, ddt_bias [D]
 * or NULL.  Nothing of the forward call is needed but its inputs.
 */
gla_status gla_scan_bwd(const void *u, int64_t u_stride, const void *dt, int64_t dt_stride,
                        const float *a, const void *b, int64_t b_stride, const void *c,
                        int64_t c_stride, const float *skip, const void *z, int64_t z_stride,
                        const float *dt_bias, const float *init_state, const void *d_out,
                        const float *d_final_state, void *du, void *ddt, float *da, void *db,
                        void *dc, float *dskip, void *dz, float *ddt_bias, float *d_init_state,
                        const int32_t *cu_seqlens, int B, int T, int D, int N, void *workspace,
                        size_t workspace_bytes, gla_stream_t stream, unsigned flags);
size_t gla_scan_bwd_workspace_size(int B, int T, int D, int N, int packed);

/*
 * gla_scan_step -- one token for each of `rows` sequences: u, dt, z, out
 * [rows, D], b, c [rows, N]; state fp32 [rows, D, N] updated in place, or a
 * pool with slots and out_slots as for gla_conv_step.
 */
gla_status gla_scan_step(const void *u, int64_t u_stride, const void *dt, int64_t dt_stride,
                         const float *a, const void *b, int64_t b_stride, const void *c,
                         int64_t c_stride, const float *skip, const void *z, int64_t z_stride,
                         const float *dt_bias, float *state, int num_slots,
                         const int32_t *slots, const int32_t *out_slots, void *out, int rows,
                         int D, int N, gla_stream_t stream, unsigned flags);

/*
 * The gated linear recurrence: one state per channel, whose decay comes from a gate of
 * the token's own.  With s(v) = 1 / (1 + exp(-v)), for every sequence and channel d
 *     log a = decay[d] s(f[t][d]);  without decay: log s(f[t][d])
 *     m     = sqrt(1 - a^2) with GLA_FLAG_UNIT_VARIANCE, else 1 - a
 *     h[t]  = a h[t-1] + m s(i[t][d]) x[t][d]            (without i: m x)
 *     out   = h[t] z s(z)                                  (without z: h[t])
 * The pages the library's recurrence comes from have no counterpart; these entry
 * points stand beside it and the scan for layers without a state matrix.
 *
 *   x, f, i, z   [rows, D]: bf16, or fp32 with GLA_FLAG_FP32_IO; row strides as for
 *                the scan; i and z may be NULL (their strides are then ignored)
 *   decay        fp32 [D], finite and <= 0 (a value above 0 acts as 0, and its gradient
 *                is 0; a channel whose decay is NaN is NaN), or NULL.
 *                1 - a is computed without cancellation, so that m is right where a rounds to
 *                1; m = sqrt(1 - a^2) and its share of the gradients are 0 where 1 - a^2,
 *                or s(f) with a decay, is below 2^-126 (the smallest normal number), in
 *                every call alike.
 *   init_state   fp32 [B, D] or NULL (zeros); final_state likewise or NULL (not
 *                written), may be init_state itself
 *   out          [rows, D], x's dtype (fp32 with GLA_FLAG_FP32_OUT)
 *   D            as for the scan; rows dense or packed (cu_seqlens) as for the scan
 * Nothing of one sequence reaches another, infinities and NaN included.  Inside
 * a sequence an infinite state stays infinite until the product of the decays
 * behind it underflows, and is NaN from then on.
 */
gla_status gla_recur_fwd(const void *x, int64_t x_stride, const void *f, int64_t f_stride,
                         const void *i, int64_t i_stride, const void *z, int64_t z_stride,
                         const float *decay, const float *init_state, void *out,
                         float *final_state, const int32_t *cu_seqlens, int B, int T, int D,
                         gla_stream_t stream, unsigned flags);

/*
 * gla_recur_bwd -- the gradient of gla_recur_fwd, from its inputs alone.  d_out
 * [rows, D] in x's dtype; d_final_state, d_init_state fp32 [B, D] or NULL; dx, df,
 * di, dz [rows, D] in x's dtype (fp32 with GLA_FLAG_FP32_OUT), di and dz NULL
 * exactly without i and z; d_decay fp32 [D] or NULL.  workspace:
 * gla_recur_bwd_workspace_size(...) bytes, 256-byte aligned.  Sums run in a
 * fixed order (the same inputs give the same bits).
 */
gla_status gla_recur_bwd(const void *x, int64_t x_stride, const void *f, int64_t f_stride,
                         const void *i, int64_t i_stride, const void *z, int64_t z_stride,
                         const float *decay, const float *init_state, const void *d_out,
                         const float *d_final_state, void *dx, void *df, void *di, void *dz,
                         float *d_decay, float *d_init_state, const int32_t *cu_seqlens, int B,
                         int T, int D, void *workspace, size_t workspace_bytes,
                         gla_stream_t stream, unsigned flags);
size_t gla_recur_bwd_workspace_size(int B, int T, int D, int packed);

/*
 * gla_recur_step -- one token for each of N sequences: x, f, i, z, out [N, D];
 * state fp32 [N, D] updated in place, or a pool with slots and out_slots as for
 * gla_conv_step.
 */
gla_status gla_recur_step(const void *x, int64_t x_stride, const void *f, int64_t f_stride,
                          const void *i, int64_t i_stride, const void *z, int64_t z_stride,
                          const float *decay, float *state, int num_slots, const int32_t *slots,
                          const int32_t *out_slots, void *out, int N, int D,
                          gla_stream_t stream, unsigned flags);

/*
 * gla_block_norm_fwd -- what stands between two blocks, for every row
 *     p = norm(y) post_weight + post_bias          (post_weight NULL: p = y)
 *     s = res + scale p z / (1 + exp(-z))          (scale, z NULL: 1; y NULL: s = res)
 *     out = norm(s) weight + bias
 * norm(v) = v / sqrt(mean(v^2) + eps), with GLA_FLAG_LAYER_NORM of v - mean(v).
 *
 *   res          [rows, D], contiguous: the residual stream, in y's dtype, or fp32
 *                with GLA_FLAG_FP32_RESIDUAL
 *   y            [rows, D] with y_stride, the block's output, bf16 (fp32 with
 *                GLA_FLAG_FP32_IO, and then everything is), or NULL; z [rows, D]
 *                with z_stride, y's dtype, or NULL.  Strides as for the scan.
 *   post_weight, post_bias, scale, weight, bias   fp32 [D], 16-byte aligned;
 *                each may be NULL (weight exactly without out; the others: left out)
 *   eps          >= 0
 *   res_out      [rows, D] in res's dtype: s, or NULL (not written; NULL without
 *                y).  May be res itself.
 *   out          [rows, D] in y's dtype (fp32 with GLA_FLAG_FP32_OUT), from the
 *                unrounded s, or NULL
 *   D            a multiple of 8, at most 8192
 * Alignment: every pointer 16 bytes.  Outputs must not overlap anything else.
 */
gla_status gla_block_norm_fwd(const void *res, const void *y, int64_t y_stride, const void *z,
                              int64_t z_stride, const float *post_weight, const float *post_bias,
                              const float *scale, const float *weight, const float *bias,
                              float eps, void *res_out, void *out, int rows, int D,
                              gla_stream_t stream, unsigned flags);

/*
 * gla_block_norm_bwd -- the gradient of gla_block_norm_fwd, from its inputs alone.
 * d_out [rows, D] in y's dtype and d_res_out [rows, D] in res's dtype, contiguous,
 * or NULL (zero).  d_out needs weight, as d_weight and d_bias do.
 * d_res [rows, D] in res's dtype, dy and dz [rows, D] in y's (all fp32 with
 * GLA_FLAG_FP32_OUT); dy NULL exactly without y, dz without z.  d_post_weight,
 * d_post_bias, d_scale, d_weight, d_bias fp32 [D], each or NULL (not computed).
 * workspace: gla_block_norm_bwd_workspace_size(...) bytes, 256-byte aligned.
 * Sums over rows run in a fixed order.
 */
gla_status gla_block_norm_bwd(const void *res, const void *y, int64_t y_stride, const void *z,
                              int64_t z_stride, const float *post_weight, const float *post_bias,
                              const float *scale, const float *weight, float eps,
                              const void *d_out, const void *d_res_out, void *d_res, void *dy,
                              void *dz, float *d_post_weight, float *d_post_bias, float *d_scale,
                              float *d_weight, float *d_bias, int rows, int D, void *workspace,
                              size_t workspace_bytes, gla_stream_t stream, unsigned flags);
size_t gla_block_norm_bwd_workspace_size(int rows, int D);

/*
 * gla_glu_fwd -- the gated feed-forward projections: g = x w_gate^T, u = x w_up^T,
 *     out = g u / (1 + exp(-g))
 *
 *   x            [rows, D] bf16 with x_stride (rows start on 16 bytes)
 *   w_gate, w_up [F, D] bf16, contiguous
 *   out          [rows, F] bf16 (fp32 with GLA_FLAG_FP32_OUT)
 *   D, F         multiples of 8, 8 to 2^20 (with rows; 0 returns GLA_ERR_UNSUPPORTED where
 *                there is something to compute); any number of rows
 * g and u are fp32 sums that stay on the chip.  fp32 inputs (GLA_FLAG_FP32_IO)
 * return GLA_ERR_UNSUPPORTED.  Alignment: every pointer 16 bytes.
 */
gla_status gla_glu_fwd(const void *x, int64_t x_stride, const void *w_gate, const void *w_up,
                       void *out, int rows, int D, int F, gla_stream_t stream, unsigned flags);

/*
 * gla_glu_bwd -- the gradient of gla_glu_fwd, from its inputs alone: with s = 1 / (1 + exp(-g))
 *     dg = d_out u s (1 + g (1 - s)),  du = d_out g s        (rounded to bf16)
 *     dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x
 * d_out [rows, F] bf16; dx [rows, D], dw_gate and dw_up [F, D], all bf16 (fp32 with
 * GLA_FLAG_FP32_OUT, of the same rounded dg and du).  workspace:
 * gla_glu_bwd_workspace_size(...) bytes, 256-byte aligned (dg and du).
 * At most 2^26 rows (more return GLA_ERR_UNSUPPORTED): dw_gate and dw_up are sums over all rows
 * in one fp32 accumulator, whose length bounds both its rounding and the time for
 * which the kernel waits for it.
 */
gla_status gla_glu_bwd(const void *x, int64_t x_stride, const void *w_gate, const void *w_up,
                       const void *d_out, void *dx, void *dw_gate, void *dw_up, int rows, int D,
                       int F, void *workspace, size_t workspace_bytes, gla_stream_t stream,
                       unsigned flags);
size_t gla_glu_bwd_workspace_size(int rows, int D, int F);

/*
 * The pages of state pools.  A sequence's state is page i of every pool (one
 * pool per layer and kind of state: the pools of gla_decode_step_slots,
 * gla_conv_step, gla_scan_step), and `used` (DEVICE int32 [num_pages]) is 0 for
 * a free page.  The operators below read and write the tables on the device,
 * in page order, and move the pages of all pools; the host waits for nothing.
 *
 *   pools        HOST array of num_pools pools (read before the call returns):
 *                page i is the page_bytes bytes at base + i * page_bytes;
 *                page_bytes a multiple of 16, at most 2^32
 *   num_pages    pages of every pool, at most GLA_MAX_PAGES
 *   used, used_out   [num_pages]; used_out may be used (in place)
 * An entry of a table that names no page it could (out of range; a free page
 * where a used one is meant) is skipped and reported by gla_status_sync as
 * GLA_ERR_INVALID_ARG.  -1 entries are skipped silently.
 */
#define GLA_MAX_PAGES 524288
#define GLA_PAGE_NEW (-2)
typedef struct gla_page_pool {
    void *base;         /* DEVICE, 16-byte aligned */
    int64_t page_bytes;
} gla_page_pool;

/*
 * gla_pages_copy -- page dst[i] = page src[i] (DEVICE int32 [n] each) for all
 * pairs at once.  A pair whose dst another pair writes, or whose dst another
 * pair reads, is skipped and reported.  copied [n] receives dst[i] for the
 * pairs that were copied and -1 for the others.
 */
gla_status gla_pages_copy(const gla_page_pool *pools, int num_pools, int num_pages,
                          const int32_t *src, const int32_t *dst, int32_t *copied, int n,
                          gla_stream_t stream);

/*
 * gla_pages_fork -- a new page for every entry of parents: a copy of page
 * parents[i] (used; several entries may name it), or, where it is
 * GLA_PAGE_NEW, zeros.  children[i] receives its number: the free pages in
 * ascending order go to the entries in order.  When no page is left an entry
 * gets -1 and the call is reported as GLA_ERR_INVALID_ARG.
 */
gla_status gla_pages_fork(const gla_page_pool *pools, int num_pools, int num_pages,
                          const int32_t *used, int32_t *used_out, const int32_t *parents,
                          int32_t *children, int n, gla_stream_t stream);

/*
 * gla_pages_compact -- with L pages used, moves the used pages at or behind L
 * to the free pages in front of L (the k-th of the ones, in ascending order,
 * to the k-th of the others), so that pages 0 .. L-1 are the used ones; the
 * rest keep their bytes.  forward [num_pages] receives every used page's new
 * number (-1 for the free pages); slots_out[i] = forward[slots[i]] (-1 for -1,
 * and for an entry that names no used page); slots_out may be slots.
 */
gla_status gla_pages_compact(const gla_page_pool *pools, int num_pools, int num_pages,
                             const int32_t *used, int32_t *used_out, const int32_t *slots,
                             int32_t *slots_out, int n, int32_t *forward, gla_stream_t stream);

/*
 * gla_pages_free -- marks the pages slots[0 .. n) free; their bytes stay.  A
 * page that was free already, or is named twice, is reported.
 */
gla_status gla_pages_free(const int32_t *used, int32_t *used_out, int num_pages,
                          const int32_t *slots, int n, gla_stream_t stream);

/* Static English text for a status code (never NULL). */
const char *gla_status_string(gla_status status);

/*
 * gla_status_sync -- wait for `stream`, then read and clear the current GPU's
 * device status word.  Returns GLA_ERR_CUDA if the stream reports a CUDA error,
 * otherwise the most severe device-side status seen since the last call
 * (GLA_ERR_TIMEOUT over GLA_ERR_UNSUPPORTED over GLA_ERR_INVALID_ARG over
 * GLA_OK).  GLA_ERR_UNSUPPORTED here means a tensor-core kernel found its
 * shared-memory window not 1024-byte aligned and wrote nothing.
 */
gla_status gla_status_sync(gla_stream_t stream);

/* Text of the calling thread's most recent failure: the CUDA error behind a
 * GLA_ERR_CUDA, or the size limit behind gla_chunk_bwd_fixed_workspace's
 * GLA_ERR_UNSUPPORTED (thread-local storage, never NULL; "no error" if there
 * was none). */
const char *gla_last_error_string(void);

/*
 * gla_set_wait_limit_ns -- the wall-time limit of the waits with which the
 * warp roles of the tensor-core prefill kernels (gla_chunk_fwd, the mixer and
 * backward calls that run them), of the projections (gla_glu_*) and of the gated
 * recurrence's prompts and gradients (gla_recur_fwd, gla_recur_bwd) hand work to
 * one another; 0 restores the default, 2 s.  Process-wide, read at each launch;
 * returns the previous setting (0 = the default).  A wait that runs out makes the
 * kernel stop issuing work, let its own copies and matrix products land (with
 * limits of their own), release its tensor memory and return: gla_status_sync
 * then reports GLA_ERR_TIMEOUT and the call's outputs are undefined.  For tests of
 * that path: a limit shorter than a chunk's hand-offs (about a microsecond) makes
 * the next prefill fail that way, and the call after the default is restored
 * runs normally.  In the projections a wait lasts as long as one tile's sum over
 * K (0.34 us for every 64), in the recurrence microseconds; its limit there is longer
 * by 4 us for each packed sequence.  The pages have no counterpart (failure
 * handling is the library's own).
 */
uint64_t gla_set_wait_limit_ns(uint64_t nanoseconds);

/* Library version, "major.minor.patch". */
const char *gla_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GLA_H_ */
