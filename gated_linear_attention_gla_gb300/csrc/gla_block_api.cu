// gla_block_api.cu -- the C ABI of the gated linear recurrence, the norms between blocks
// and the gated feed-forward projections: argument checks and dispatch.  As in
// gla_api.cu every check runs on the host before anything is enqueued; device
// arrays (cu_seqlens, slots) are checked by the kernels.
#include "gla.h"
#include "gla_checks.cuh"
#include "gla_internal.cuh"

using namespace gla::checks;

extern "C" {

// ------------------------------------------------------------------ norms between blocks
static gla_status norm_args(const void* res, const void* y, int64_t y_stride, const void* z,
                            int64_t z_stride, const float* post_weight, const float* post_bias,
                            const float* scale, const float* weight, float eps, int rows, int D,
                            unsigned flags, gla::NormArgs* a) {
  constexpr unsigned known = GLA_FLAG_FP32_IO | GLA_FLAG_FP32_OUT | GLA_FLAG_FP32_RESIDUAL |
                             GLA_FLAG_LAYER_NORM;
  if ((flags & ~known) != 0u || rows < 0 || D < 0 || !(eps >= 0.f) || eps > 3.4e38f)
    return GLA_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > gla::kNormMaxD) return GLA_ERR_UNSUPPORTED;
  const bool fp32 = (flags & GLA_FLAG_FP32_IO) != 0;
  const long long esz = fp32 ? 4 : 2;
  if (rows > 0 && !y && (z || post_weight || scale)) return GLA_ERR_INVALID_ARG;
  if (!post_weight && post_bias) return GLA_ERR_INVALID_ARG;
  if (D > 0 && ((y && (stride_bad(y_stride, D) || too_many(rows, y_stride))) ||
                (z && (stride_bad(z_stride, D) || too_many(rows, z_stride)))))
    return GLA_ERR_INVALID_ARG;
  if (rows > 0 && D > 0 && !res) return GLA_ERR_INVALID_ARG;
  if (!aligned(res, 16) || !aligned(y, 16) || !aligned(z, 16) || !aligned(post_weight, 16) ||
      !aligned(post_bias, 16) || !aligned(scale, 16) || !aligned(weight, 16) ||
      (y && stride_misaligned(y_stride, esz)) || (z && stride_misaligned(z_stride, esz)))
    return GLA_ERR_MISALIGNED;
  a->res = res; a->y = y; a->z = z; a->y_stride = y_stride; a->z_stride = z_stride;
  a->post_weight = post_weight; a->post_bias = post_bias; a->scale = scale; a->weight = weight;
  a->eps = eps; a->inv_d = D > 0 ? 1.f / D : 0.f; a->rows = rows; a->D = D;
  a->layer = (flags & GLA_FLAG_LAYER_NORM) != 0; a->fp32_io = fp32;
  a->fp32_res = fp32 || (flags & GLA_FLAG_FP32_RESIDUAL) != 0;
  a->fp32_out = fp32 || (flags & GLA_FLAG_FP32_OUT) != 0;
  return GLA_OK;
}

gla_status gla_block_norm_fwd(const void* res, const void* y, int64_t y_stride, const void* z,
                              int64_t z_stride, const float* post_weight, const float* post_bias,
                              const float* scale, const float* weight, const float* bias,
                              float eps, void* res_out, void* out, int rows, int D,
                              gla_stream_t stream, unsigned flags) {
  gla::NormArgs a{};
  const gla_status bad = norm_args(res, y, y_stride, z, z_stride, post_weight, post_bias, scale,
                                   weight, eps, rows, D, flags, &a);
  if (bad != GLA_OK) return bad;
  if (rows == 0 || D == 0) return GLA_OK;  // (pointers of empty tensors are null)
  if ((!y && res_out) || (out && !weight) || (!out && (weight || bias)))
    return GLA_ERR_INVALID_ARG;
  if (!res_out && !out) return GLA_ERR_INVALID_ARG;
  if (!aligned(bias, 16) || !aligned(res_out, 16) || !aligned(out, 16)) return GLA_ERR_MISALIGNED;
  const long long esz = a.fp32_io ? 4 : 2, rsz = a.fp32_res ? 4 : 2, osz = a.fp32_out ? 4 : 2;
  const long long n = (long long)rows * D;
  const size_t vec = (size_t)D * 4;
  const Range in[] = {{res == res_out ? nullptr : res, (size_t)(n * rsz)},
                      {y, y ? span(rows, y_stride, D, esz) : 0},
                      {z, z ? span(rows, z_stride, D, esz) : 0},
                      {post_weight, vec}, {post_bias, vec}, {scale, vec}, {weight, vec}, {bias, vec}};
  const Range outs[] = {{res_out, (size_t)(n * rsz)}, {out, (size_t)(n * osz)}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  a.bias = bias; a.res_out = res_out; a.out = out;
  return finish(gla::launch_norm_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gla_block_norm_bwd_workspace_size(int rows, int D) {
  if (rows < 0 || D <= 0 || D % 8 != 0 || D > gla::kNormMaxD) return 0;
  return gla::norm_bwd_workspace(rows, D);
}

gla_status gla_block_norm_bwd(const void* res, const void* y, int64_t y_stride, const void* z,
                              int64_t z_stride, const float* post_weight, const float* post_bias,
                              const float* scale, const float* weight, float eps,
                              const void* d_out, const void* d_res_out, void* d_res, void* dy,
                              void* dz, float* d_post_weight, float* d_post_bias, float* d_scale,
                              float* d_weight, float* d_bias, int rows, int D, void* workspace,
                              size_t workspace_bytes, gla_stream_t stream, unsigned flags) {
  gla::NormBwdArgs b{};
  const gla_status bad = norm_args(res, y, y_stride, z, z_stride, post_weight, post_bias, scale,
                                   weight, eps, rows, D, flags, &b.f);
  if (bad != GLA_OK) return bad;
  if (D == 0) return GLA_OK;
  if ((!weight && (d_out || d_weight || d_bias)) ||
      (!post_weight && (d_post_weight || d_post_bias)) || (!post_bias && d_post_bias) ||
      (!scale && d_scale) || (!y && dy) || (!z && dz) ||
      (rows > 0 && (!d_res || (y && !dy) || (z && !dz))))
    return GLA_ERR_INVALID_ARG;
  if (!aligned(d_out, 16) || !aligned(d_res_out, 16) || !aligned(d_res, 16) || !aligned(dy, 16) ||
      !aligned(dz, 16) || !aligned(d_post_weight, 4) || !aligned(d_post_bias, 4) ||
      !aligned(d_scale, 4) || !aligned(d_weight, 4) || !aligned(d_bias, 4) ||
      !aligned(workspace, 256))
    return GLA_ERR_MISALIGNED;
  const size_t need = gla::norm_bwd_workspace(rows, D);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GLA_ERR_INVALID_ARG;
  const gla::NormArgs& a = b.f;
  const long long esz = a.fp32_io ? 4 : 2, rsz = a.fp32_res ? 4 : 2;
  const long long gsz = a.fp32_out ? 4 : 2, grsz = a.fp32_out || a.fp32_res ? 4 : 2;
  const long long n = (long long)rows * D;
  const size_t vec = (size_t)D * 4;
  const Range in[] = {{res, (size_t)(n * rsz)},
                      {y, y ? span(rows, y_stride, D, esz) : 0},
                      {z, z ? span(rows, z_stride, D, esz) : 0},
                      {post_weight, vec}, {post_bias, vec}, {scale, vec}, {weight, vec},
                      {d_out, (size_t)(n * esz)}, {d_res_out, (size_t)(n * rsz)}};
  const Range outs[] = {{d_res, (size_t)(n * grsz)}, {dy, (size_t)(n * gsz)},
                        {dz, (size_t)(n * gsz)}, {d_post_weight, vec}, {d_post_bias, vec},
                        {d_scale, vec}, {d_weight, vec}, {d_bias, vec}, {workspace, need}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  b.d_out = d_out; b.d_res_out = d_res_out; b.d_res = d_res; b.dy = dy; b.dz = dz;
  b.d_post_weight = d_post_weight; b.d_post_bias = d_post_bias; b.d_scale = d_scale;
  b.d_weight = d_weight; b.d_bias = d_bias;
  return finish(gla::launch_norm_bwd(b, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ gated linear recurrence
static constexpr unsigned kRecurFlags =
    GLA_FLAG_FP32_IO | GLA_FLAG_FP32_OUT | GLA_FLAG_UNIT_VARIANCE;

// The rows shared by the three entry points; `rows` of them.
static gla_status recur_rows(const void* x, int64_t x_stride, const void* f, int64_t f_stride,
                             const void* i, int64_t i_stride, const void* z, int64_t z_stride,
                             const float* decay, long long rows, int D, unsigned flags) {
  const long long esz = (flags & GLA_FLAG_FP32_IO) ? 4 : 2;
  if (stride_bad(x_stride, D) || stride_bad(f_stride, D) || (i && stride_bad(i_stride, D)) ||
      (z && stride_bad(z_stride, D)) || too_many(rows, x_stride) || too_many(rows, f_stride) ||
      (i && too_many(rows, i_stride)) || (z && too_many(rows, z_stride)) || (rows > 0 && (!x || !f)))
    return GLA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(f, 16) || !aligned(i, 16) || !aligned(z, 16) ||
      stride_misaligned(x_stride, esz) || stride_misaligned(f_stride, esz) ||
      (i && stride_misaligned(i_stride, esz)) || (z && stride_misaligned(z_stride, esz)) ||
      !aligned(decay, 16))
    return GLA_ERR_MISALIGNED;
  return GLA_OK;
}

// Limit of a wait inside the recurrence's kernels.  Warps look through packed offsets (all of them for
// malformed and empty ones, runs of empty ones between two rows) while others wait for their
// maps: at most some dependent reads a sequence.
static uint64_t recur_wait_ns(const int32_t* cu_seqlens, int B) {
  const uint64_t limit = gla::handoff_wait_limit_ns(), more = cu_seqlens ? 4000ull * (uint64_t)B : 0;
  return limit + more < limit ? ~0ull : limit + more;
}

#define GLA_RECUR_INPUTS(rows, esz)                                                          \
  {x, span(rows, x_stride, D, esz)}, {f, span(rows, f_stride, D, esz)},                       \
      {i, i ? span(rows, i_stride, D, esz) : 0}, {z, z ? span(rows, z_stride, D, esz) : 0},   \
      {decay, (size_t)D * 4}

gla_status gla_recur_fwd(const void* x, int64_t x_stride, const void* f, int64_t f_stride,
                         const void* i, int64_t i_stride, const void* z, int64_t z_stride,
                         const float* decay, const float* init_state, void* out,
                         float* final_state, const int32_t* cu_seqlens, int B, int T, int D,
                         gla_stream_t stream, unsigned flags) {
  if ((flags & ~kRecurFlags) != 0u || B < 0 || T < 0 || D < 0) return GLA_ERR_INVALID_ARG;
  if (!channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (B == 0 || D == 0) return GLA_OK;
  const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
  const long long st = (long long)B * D;
  if (st > kMaxElems || (!cu_seqlens && ((long long)D + 63) / 64 * B > kMaxGrid))
    return GLA_ERR_INVALID_ARG;
  const gla_status bad = recur_rows(x, x_stride, f, f_stride, i, i_stride, z, z_stride, decay,
                                    rows, D, flags);
  if (bad != GLA_OK) return bad;
  if (rows > 0 && !out) return GLA_ERR_INVALID_ARG;
  if (rows == 0 && !final_state) return GLA_OK;
  if (!aligned(init_state, 16) || !aligned(out, 16) || !aligned(final_state, 16) ||
      !aligned(cu_seqlens, 4))
    return GLA_ERR_MISALIGNED;
  const bool fp32 = (flags & GLA_FLAG_FP32_IO) != 0;
  const bool f32out = fp32 || (flags & GLA_FLAG_FP32_OUT) != 0;
  const long long esz = fp32 ? 4 : 2, osz = f32out ? 4 : 2;
  const Range in[] = {GLA_RECUR_INPUTS(rows, esz),
                      {init_state == final_state ? nullptr : init_state, (size_t)st * 4},
                      {cu_seqlens, ((size_t)B + 1) * 4}};
  const Range outs[] = {{out, (size_t)(rows * D * osz)}, {final_state, (size_t)st * 4}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  gla::RecurArgs a{};
  a.status = gla::device_status_word(&err);
  if (!a.status) return finish(err);
  a.x = x; a.f = f; a.i = i; a.z = z; a.x_stride = x_stride; a.f_stride = f_stride;
  a.i_stride = i_stride; a.z_stride = z_stride; a.decay = decay; a.init_state = init_state;
  a.out = out; a.final_state = final_state; a.cu_seqlens = cu_seqlens;
  a.B = B; a.T = T; a.D = D; a.unit = (flags & GLA_FLAG_UNIT_VARIANCE) != 0;
  a.fp32_io = fp32; a.fp32_out = f32out; a.wait_ns = recur_wait_ns(cu_seqlens, B);
  return finish(gla::launch_recur_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gla_recur_bwd_workspace_size(int B, int T, int D, int packed) {
  if (B < 0 || T < 0 || D <= 0 || !channels_ok(D)) return 0;
  return gla::recur_bwd_workspace(B, packed ? (long long)T : (long long)B * T, D, packed != 0);
}

gla_status gla_recur_bwd(const void* x, int64_t x_stride, const void* f, int64_t f_stride,
                         const void* i, int64_t i_stride, const void* z, int64_t z_stride,
                         const float* decay, const float* init_state, const void* d_out,
                         const float* d_final_state, void* dx, void* df, void* di, void* dz,
                         float* d_decay, float* d_init_state, const int32_t* cu_seqlens, int B,
                         int T, int D, void* workspace, size_t workspace_bytes,
                         gla_stream_t stream, unsigned flags) {
  if ((flags & ~kRecurFlags) != 0u || B < 0 || T < 0 || D < 0) return GLA_ERR_INVALID_ARG;
  if (!channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (D == 0) return GLA_OK;
  const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
  const long long st = (long long)B * D;
  if (st > kMaxElems || (!cu_seqlens && ((long long)D + 63) / 64 * B > kMaxGrid))
    return GLA_ERR_INVALID_ARG;
  const gla_status bad = recur_rows(x, x_stride, f, f_stride, i, i_stride, z, z_stride, decay,
                                    rows, D, flags);
  if (bad != GLA_OK) return bad;
  if ((rows > 0 && (B == 0 || !d_out || !dx || !df || (i && !di) || (z && !dz))) || (!i && di) ||
      (!z && dz) || (!decay && d_decay))
    return GLA_ERR_INVALID_ARG;
  if (!aligned(init_state, 16) || !aligned(d_out, 16) || !aligned(d_final_state, 16) ||
      !aligned(dx, 16) || !aligned(df, 16) || !aligned(di, 16) || !aligned(dz, 16) ||
      !aligned(d_decay, 4) || !aligned(d_init_state, 16) || !aligned(cu_seqlens, 4) ||
      !aligned(workspace, 256))
    return GLA_ERR_MISALIGNED;
  const size_t need = gla::recur_bwd_workspace(B, rows, D, cu_seqlens != nullptr);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GLA_ERR_INVALID_ARG;
  const bool fp32 = (flags & GLA_FLAG_FP32_IO) != 0;
  const bool f32out = fp32 || (flags & GLA_FLAG_FP32_OUT) != 0;
  const long long esz = fp32 ? 4 : 2, osz = f32out ? 4 : 2;
  const size_t grad = (size_t)(rows * D * osz);
  const Range in[] = {GLA_RECUR_INPUTS(rows, esz),
                      {init_state, (size_t)st * 4},
                      {d_out, (size_t)(rows * D * esz)},
                      {d_final_state, (size_t)st * 4},
                      {cu_seqlens, ((size_t)B + 1) * 4}};
  const Range outs[] = {{dx, grad}, {df, grad}, {di, grad}, {dz, grad}, {d_decay, (size_t)D * 4},
                        {d_init_state, (size_t)st * 4}, {workspace, need}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  gla::RecurBwdArgs g{};
  gla::RecurArgs& a = g.f;
  a.status = gla::device_status_word(&err);
  if (!a.status) return finish(err);
  a.x = x; a.f = f; a.i = i; a.z = z; a.x_stride = x_stride; a.f_stride = f_stride;
  a.i_stride = i_stride; a.z_stride = z_stride; a.decay = decay; a.init_state = init_state;
  a.cu_seqlens = cu_seqlens; a.B = B; a.T = T; a.D = D;
  a.unit = (flags & GLA_FLAG_UNIT_VARIANCE) != 0; a.fp32_io = fp32; a.fp32_out = f32out;
  a.wait_ns = recur_wait_ns(cu_seqlens, B);
  g.d_out = d_out; g.d_final_state = d_final_state; g.dx = dx; g.df = df; g.di = di; g.dz = dz;
  g.d_decay = d_decay; g.d_init_state = d_init_state;
  return finish(gla::launch_recur_bwd(g, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

gla_status gla_recur_step(const void* x, int64_t x_stride, const void* f, int64_t f_stride,
                          const void* i, int64_t i_stride, const void* z, int64_t z_stride,
                          const float* decay, float* state, int num_slots, const int32_t* slots,
                          const int32_t* out_slots, void* out, int N, int D,
                          gla_stream_t stream, unsigned flags) {
  if ((flags & ~kRecurFlags) != 0u || N < 0 || D < 0 || num_slots < 0 ||
      (!slots && (num_slots != 0 || out_slots)))
    return GLA_ERR_INVALID_ARG;
  if (!channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (N == 0 || D == 0) return GLA_OK;
  const long long pages = slots ? num_slots : N;
  if (pages * D > kMaxElems) return GLA_ERR_INVALID_ARG;
  const gla_status bad = recur_rows(x, x_stride, f, f_stride, i, i_stride, z, z_stride, decay, N,
                                    D, flags);
  if (bad != GLA_OK) return bad;
  if ((!state && pages > 0) || !out) return GLA_ERR_INVALID_ARG;
  if (!aligned(state, 16) || !aligned(out, 16) || !aligned(slots, 4) || !aligned(out_slots, 4))
    return GLA_ERR_MISALIGNED;
  const bool fp32 = (flags & GLA_FLAG_FP32_IO) != 0;
  const bool f32out = fp32 || (flags & GLA_FLAG_FP32_OUT) != 0;
  const long long esz = fp32 ? 4 : 2, osz = f32out ? 4 : 2;
  const Range in[] = {GLA_RECUR_INPUTS(N, esz), {slots, (size_t)N * 4}, {out_slots, (size_t)N * 4}};
  const Range outs[] = {{out, (size_t)((long long)N * D * osz)}, {state, (size_t)(pages * D) * 4}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  gla::RecurStepArgs a{};
  a.status = gla::device_status_word(&err);
  if (!a.status) return finish(err);
  a.x = x; a.f = f; a.i = i; a.z = z; a.x_stride = x_stride; a.f_stride = f_stride;
  a.i_stride = i_stride; a.z_stride = z_stride; a.decay = decay; a.state = state;
  a.num_slots = num_slots; a.slots = slots; a.out_slots = out_slots; a.out = out; a.N = N;
  a.D = D; a.unit = (flags & GLA_FLAG_UNIT_VARIANCE) != 0; a.fp32_io = fp32; a.fp32_out = f32out;
  return finish(gla::launch_recur_step(a, reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ gated feed-forward
static gla_status glu_args(const void* x, int64_t x_stride, const void* w_gate, const void* w_up,
                           int rows, int D, int F, unsigned flags, gla::GluArgs* a) {
  if ((flags & ~(GLA_FLAG_FP32_IO | GLA_FLAG_FP32_OUT)) != 0u || rows < 0 || D < 0 || F < 0)
    return GLA_ERR_INVALID_ARG;
  if ((flags & GLA_FLAG_FP32_IO) || D % 8 != 0 || F % 8 != 0 || D > 1 << 20 || F > 1 << 20)
    return GLA_ERR_UNSUPPORTED;
  if (D == 0 || F == 0) return GLA_OK;
  if (stride_bad(x_stride, D) || too_many(rows, x_stride) || too_many(rows, F) ||
      !w_gate || !w_up || (rows > 0 && !x))
    return GLA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || stride_misaligned(x_stride, 2) || !aligned(w_gate, 16) ||
      !aligned(w_up, 16))
    return GLA_ERR_MISALIGNED;
  a->x = x; a->x_stride = x_stride; a->w_gate = w_gate; a->w_up = w_up;
  a->rows = rows; a->D = D; a->F = F; a->fp32_out = (flags & GLA_FLAG_FP32_OUT) != 0;
  return GLA_OK;
}

gla_status gla_glu_fwd(const void* x, int64_t x_stride, const void* w_gate, const void* w_up,
                       void* out, int rows, int D, int F, gla_stream_t stream, unsigned flags) {
  gla::GluArgs a{};
  const gla_status bad = glu_args(x, x_stride, w_gate, w_up, rows, D, F, flags, &a);
  if (bad != GLA_OK) return bad;
  if (rows == 0 || F == 0) return GLA_OK;
  if (D == 0) return GLA_ERR_UNSUPPORTED;
  if (!out) return GLA_ERR_INVALID_ARG;
  if (!aligned(out, 16)) return GLA_ERR_MISALIGNED;
  const size_t w = (size_t)F * D * 2;
  const Range in[] = {{x, span(rows, x_stride, D, 2)}, {w_gate, w}, {w_up, w}};
  const Range outs[] = {{out, (size_t)rows * F * (a.fp32_out ? 4 : 2)}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  a.status = gla::device_status_word(&err);
  if (!a.status) return finish(err);
  a.out = out;
  return finish(gla::launch_glu_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gla_glu_bwd_workspace_size(int rows, int D, int F) {
  if (rows <= 0 || rows > gla::kGluBwdMaxRows || D <= 0 || F <= 0) return 0;
  return gla::glu_bwd_workspace(rows, D, F);
}

gla_status gla_glu_bwd(const void* x, int64_t x_stride, const void* w_gate, const void* w_up,
                       const void* d_out, void* dx, void* dw_gate, void* dw_up, int rows, int D,
                       int F, void* workspace, size_t workspace_bytes, gla_stream_t stream,
                       unsigned flags) {
  gla::GluBwdArgs b{};
  const gla_status bad = glu_args(x, x_stride, w_gate, w_up, rows, D, F, flags, &b.f);
  if (bad != GLA_OK) return bad;
  if (rows > gla::kGluBwdMaxRows) return GLA_ERR_UNSUPPORTED;
  if (D == 0) return GLA_OK;
  if (F == 0) return rows == 0 ? GLA_OK : GLA_ERR_UNSUPPORTED;
  if (!dw_gate || !dw_up || (rows > 0 && (!d_out || !dx))) return GLA_ERR_INVALID_ARG;
  if (!aligned(d_out, 16) || !aligned(dx, 16) || !aligned(dw_gate, 16) || !aligned(dw_up, 16) ||
      !aligned(workspace, 256))
    return GLA_ERR_MISALIGNED;
  const size_t need = rows > 0 ? gla::glu_bwd_workspace(rows, D, F) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GLA_ERR_INVALID_ARG;
  const size_t w = (size_t)F * D * 2, gsz = b.f.fp32_out ? 4 : 2;
  const Range in[] = {{x, span(rows, x_stride, D, 2)}, {w_gate, w}, {w_up, w},
                      {d_out, (size_t)rows * F * 2}};
  const Range outs[] = {{dx, (size_t)rows * D * gsz}, {dw_gate, (size_t)F * D * gsz},
                        {dw_up, (size_t)F * D * gsz}, {workspace, need}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  b.f.status = gla::device_status_word(&err);
  if (!b.f.status) return finish(err);
  b.d_out = d_out; b.dx = dx; b.dw_gate = dw_gate; b.dw_up = dw_up;
  return finish(gla::launch_glu_bwd(b, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
