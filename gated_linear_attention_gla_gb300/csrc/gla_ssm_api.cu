// gla_ssm_api.cu -- the C ABI of the causal convolution, the selective scan and
// the page operators: argument checks and dispatch.  As in gla_api.cu every
// check runs on the host before anything is enqueued; device arrays
// (cu_seqlens, slots, page tables) are checked by the kernels.
#include <cmath>
#include <cstdint>

#include "gla.h"
#include "gla_internal.cuh"

namespace {

constexpr long long kMaxElems = 1ll << 40;  // per tensor; keeps index arithmetic exact
constexpr long long kMaxGrid = 0x7fffffffll;

static_assert(GLA_PAGE_NEW == gla::kPageNew && GLA_MAX_PAGES == gla::kMaxPages,
              "the header states the kernels' constants");

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// A byte range of a call's arguments.
struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// every output apart from every input and from the other outputs
template <int I, int O> bool disjoint(const Range (&in)[I], const Range (&out)[O]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (overlap(out[o], in[i])) return false;
    for (int o2 = o + 1; o2 < O; ++o2)
      if (overlap(out[o], out[o2])) return false;
  }
  return true;
}

// Bytes spanned by `rows` rows of `cols` elements, `stride` elements apart.
size_t span(long long rows, long long stride, long long cols, long long esz) {
  return rows > 0 ? (size_t)(((rows - 1) * stride + cols) * esz) : 0;
}

gla_status finish(cudaError_t e) { return static_cast<gla_status>(gla::cuda_result(e)); }

bool ns_ok(int n) { return n == 8 || n == 16 || n == 32 || n == 64; }
bool channels_ok(int D) { return D % 8 == 0 && D <= 1 << 24; }

// Rows, channel count and row strides shared by the entry points below.
// stride rows must hold the columns and keep every row 16-byte aligned.
bool stride_bad(long long stride, int cols) { return stride < cols || stride > kMaxElems; }
bool stride_misaligned(long long stride, long long esz) { return stride * esz % 16 != 0; }

}  // namespace

extern "C" {

gla_status gla_conv_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias,
                        const void* init_state, void* out, void* final_state,
                        const int32_t* cu_seqlens, int B, int T, int D, int W,
                        gla_stream_t stream, unsigned flags) {
  if ((flags & ~(GLA_FLAG_FP32_IO | GLA_FLAG_FP32_OUT | GLA_FLAG_SILU)) != 0u || B < 0 || T < 0 ||
      D < 0)
    return GLA_ERR_INVALID_ARG;
  if (W < 2 || W > 4 || !channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (B == 0 || D == 0) return GLA_OK;
  const bool fp32 = (flags & GLA_FLAG_FP32_IO) != 0;
  const bool f32out = fp32 || (flags & GLA_FLAG_FP32_OUT) != 0;
  const long long esz = fp32 ? 4 : 2, osz = f32out ? 4 : 2;
  const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
  if (stride_bad(x_stride, D) || rows * x_stride > kMaxElems ||
      (long long)B * (W - 1) * D > kMaxElems || (rows + 7) / 8 + B > kMaxGrid)
    return GLA_ERR_INVALID_ARG;
  if (!weight || (rows > 0 && (!x || !out))) return GLA_ERR_INVALID_ARG;
  if (rows == 0 && !final_state) return GLA_OK;
  if (!aligned(x, 16) || stride_misaligned(x_stride, esz) || !aligned(init_state, 16) ||
      !aligned(out, 16) || !aligned(final_state, 16) || !aligned(weight, 16) || !aligned(bias, 16) ||
      !aligned(cu_seqlens, 4))
    return GLA_ERR_MISALIGNED;
  const size_t st = (size_t)((long long)B * (W - 1) * D * esz);
  const Range in[] = {{x, span(rows, x_stride, D, esz)},
                      {weight, (size_t)D * W * 4},
                      {bias, (size_t)D * 4},
                      {init_state == final_state ? nullptr : init_state, st},
                      {cu_seqlens, ((size_t)B + 1) * 4}};
  const Range outs[] = {{out, (size_t)(rows * D * osz)}, {final_state, st}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  unsigned* status = gla::device_status_word(&err);
  if (!status) return finish(err);
  gla::ConvArgs a{};
  a.x = x; a.x_stride = x_stride; a.weight = weight; a.bias = bias;
  a.init_state = init_state; a.out = out; a.final_state = final_state;
  a.cu_seqlens = cu_seqlens; a.B = B; a.T = T; a.D = D; a.W = W;
  a.silu = (flags & GLA_FLAG_SILU) != 0; a.fp32_io = fp32; a.fp32_out = f32out;
  a.status = status;
  return finish(gla::launch_conv_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gla_conv_bwd_workspace_size(int B, int T, int D, int W, int packed) {
  if (B <= 0 || T < 0 || D <= 0 || W < 2 || W > 4) return 0;
  return gla::conv_bwd_workspace(packed ? (long long)T : (long long)B * T, D, W);
}

gla_status gla_conv_bwd(const void* x, int64_t x_stride, const float* weight, const float* bias,
                        const void* init_state, const void* d_out, const float* d_final_state,
                        void* dx, float* d_weight, float* d_bias, float* d_init_state,
                        const int32_t* cu_seqlens, int B, int T, int D, int W, void* workspace,
                        size_t workspace_bytes, gla_stream_t stream, unsigned flags) {
  if ((flags & ~(GLA_FLAG_FP32_IO | GLA_FLAG_FP32_OUT | GLA_FLAG_SILU)) != 0u || B < 0 || T < 0 ||
      D < 0)
    return GLA_ERR_INVALID_ARG;
  if (W < 2 || W > 4 || !channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (D == 0) return GLA_OK;
  const bool fp32 = (flags & GLA_FLAG_FP32_IO) != 0;
  const bool f32out = fp32 || (flags & GLA_FLAG_FP32_OUT) != 0;
  const long long esz = fp32 ? 4 : 2, osz = f32out ? 4 : 2;
  const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
  if (stride_bad(x_stride, D) || rows * x_stride > kMaxElems ||
      (long long)B * (W - 1) * D > kMaxElems || (rows + 7) / 8 + B > kMaxGrid)
    return GLA_ERR_INVALID_ARG;
  if (!weight || !d_weight || (rows > 0 && (!x || !d_out || !dx || B == 0)))
    return GLA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || stride_misaligned(x_stride, esz) || !aligned(init_state, 16) ||
      !aligned(d_out, 16) || !aligned(d_final_state, 16) || !aligned(dx, 16) ||
      !aligned(d_init_state, 16) || !aligned(weight, 16) || !aligned(bias, 16) ||
      !aligned(d_weight, 4) || !aligned(d_bias, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(workspace, 256))
    return GLA_ERR_MISALIGNED;
  const size_t need = gla::conv_bwd_workspace(rows, D, W);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GLA_ERR_INVALID_ARG;
  const long long st = (long long)B * (W - 1) * D;
  const Range in[] = {{x, span(rows, x_stride, D, esz)},
                      {weight, (size_t)D * W * 4},
                      {bias, (size_t)D * 4},
                      {init_state, (size_t)(st * esz)},
                      {d_out, (size_t)(rows * D * esz)},
                      {d_final_state, (size_t)st * 4},
                      {cu_seqlens, ((size_t)B + 1) * 4}};
  const Range outs[] = {{dx, (size_t)(rows * D * osz)},
                        {d_weight, (size_t)D * W * 4},
                        {d_bias, (size_t)D * 4},
                        {d_init_state, (size_t)st * 4},
                        {workspace, need}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  unsigned* status = gla::device_status_word(&err);
  if (!status) return finish(err);
  gla::ConvBwdArgs a{};
  a.x = x; a.x_stride = x_stride; a.weight = weight; a.bias = bias;
  a.init_state = init_state; a.d_out = d_out; a.d_final_state = d_final_state;
  a.dx = dx; a.d_weight = d_weight; a.d_bias = d_bias; a.d_init_state = d_init_state;
  a.cu_seqlens = cu_seqlens; a.B = B; a.T = T; a.D = D; a.W = W;
  a.silu = (flags & GLA_FLAG_SILU) != 0; a.fp32_io = fp32; a.fp32_out = f32out;
  a.status = status;
  return finish(gla::launch_conv_bwd(a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

gla_status gla_conv_step(const void* x, int64_t x_stride, const float* weight, const float* bias,
                         void* state, int num_slots, const int32_t* slots,
                         const int32_t* out_slots, void* out, int N, int D, int W,
                         gla_stream_t stream, unsigned flags) {
  if ((flags & ~(GLA_FLAG_FP32_IO | GLA_FLAG_FP32_OUT | GLA_FLAG_SILU)) != 0u || N < 0 || D < 0 ||
      num_slots < 0 || (!slots && (num_slots != 0 || out_slots)))
    return GLA_ERR_INVALID_ARG;
  if (W < 2 || W > 4 || !channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (N == 0 || D == 0) return GLA_OK;
  const bool fp32 = (flags & GLA_FLAG_FP32_IO) != 0;
  const bool f32out = fp32 || (flags & GLA_FLAG_FP32_OUT) != 0;
  const long long esz = fp32 ? 4 : 2, osz = f32out ? 4 : 2;
  const long long pages = slots ? num_slots : N;
  if (stride_bad(x_stride, D) || (long long)N * x_stride > kMaxElems ||
      pages * (W - 1) * D > kMaxElems)
    return GLA_ERR_INVALID_ARG;
  if (!x || !weight || (!state && pages > 0) || !out) return GLA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || stride_misaligned(x_stride, esz) || !aligned(state, 16) ||
      !aligned(out, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(slots, 4) ||
      !aligned(out_slots, 4))
    return GLA_ERR_MISALIGNED;
  const Range in[] = {{x, span(N, x_stride, D, esz)},
                      {weight, (size_t)D * W * 4},
                      {bias, (size_t)D * 4},
                      {slots, (size_t)N * 4},
                      {out_slots, (size_t)N * 4}};
  const Range outs[] = {{out, (size_t)((long long)N * D * osz)},
                        {state, (size_t)(pages * (W - 1) * D * esz)}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  unsigned* status = gla::device_status_word(&err);
  if (!status) return finish(err);
  gla::ConvStepArgs a{};
  a.x = x; a.x_stride = x_stride; a.weight = weight; a.bias = bias; a.state = state;
  a.num_slots = num_slots; a.slots = slots; a.out_slots = out_slots; a.out = out;
  a.N = N; a.D = D; a.W = W; a.silu = (flags & GLA_FLAG_SILU) != 0;
  a.fp32_io = fp32; a.fp32_out = f32out; a.status = status;
  return finish(gla::launch_conv_step(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// The checks gla_scan_fwd and gla_scan_bwd share; GLA_OK and *a filled.
gla_status scan_args(const void* u, int64_t u_stride, const void* dt, int64_t dt_stride,
                     const float* a, const void* b, int64_t b_stride, const void* c,
                     int64_t c_stride, const float* skip, const void* z, int64_t z_stride,
                     const float* dt_bias, const float* init_state, const int32_t* cu_seqlens,
                     int B, int T, int D, int N, unsigned flags, gla::ScanArgs* s) {
  const bool fp32 = (flags & GLA_FLAG_FP32_IO) != 0;
  const long long esz = fp32 ? 4 : 2;
  const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
  if (stride_bad(u_stride, D) || stride_bad(dt_stride, D) || stride_bad(b_stride, N) ||
      stride_bad(c_stride, N) || (z && stride_bad(z_stride, D)))
    return GLA_ERR_INVALID_ARG;
  const long long widest = u_stride > dt_stride ? u_stride : dt_stride;
  const long long narrow = b_stride > c_stride ? b_stride : c_stride;
  if (rows * widest > kMaxElems || rows * narrow > kMaxElems || (z && rows * z_stride > kMaxElems) ||
      (long long)B * D * N > kMaxElems || (rows / 64 + B) * (((long long)D * N + 1023) / 1024) > kMaxGrid ||
      rows * 2 * N / 256 > kMaxGrid)
    return GLA_ERR_INVALID_ARG;
  if (!a || (rows > 0 && (!u || !dt || !b || !c))) return GLA_ERR_INVALID_ARG;
  if (!aligned(u, 16) || !aligned(dt, 16) || !aligned(z, 16) || !aligned(a, 16) ||
      stride_misaligned(u_stride, esz) || stride_misaligned(dt_stride, esz) ||
      (z && stride_misaligned(z_stride, esz)) || !aligned(b, esz) || !aligned(c, esz) ||
      !aligned(skip, 4) || !aligned(dt_bias, 4) || !aligned(init_state, 16) ||
      !aligned(cu_seqlens, 4))
    return GLA_ERR_MISALIGNED;
  s->u = u; s->dt = dt; s->b = b; s->c = c; s->z = z;
  s->u_stride = u_stride; s->dt_stride = dt_stride; s->b_stride = b_stride;
  s->c_stride = c_stride; s->z_stride = z_stride;
  s->a = a; s->skip = skip; s->dt_bias = dt_bias; s->init_state = init_state;
  s->cu_seqlens = cu_seqlens; s->B = B; s->T = T; s->D = D; s->NS = N;
  s->softplus = (flags & GLA_FLAG_SOFTPLUS) != 0; s->fp32_io = fp32;
  s->fp32_out = fp32 || (flags & GLA_FLAG_FP32_OUT) != 0;
  return GLA_OK;
}

// The forward's inputs as byte ranges (init_state apart).
#define GLA_SCAN_INPUTS(s, rows, esz)                                                       \
  {s.u, span(rows, s.u_stride, s.D, esz)}, {s.dt, span(rows, s.dt_stride, s.D, esz)},        \
      {s.b, span(rows, s.b_stride, s.NS, esz)}, {s.c, span(rows, s.c_stride, s.NS, esz)},    \
      {s.z, s.z ? span(rows, s.z_stride, s.D, esz) : 0}, {s.a, (size_t)s.D * s.NS * 4},      \
      {s.skip, (size_t)s.D * 4}, {s.dt_bias, (size_t)s.D * 4},                               \
      {s.cu_seqlens, ((size_t)s.B + 1) * 4}

constexpr unsigned kScanFlags = GLA_FLAG_FP32_IO | GLA_FLAG_FP32_OUT | GLA_FLAG_SOFTPLUS;

}  // namespace

extern "C" {

size_t gla_scan_fwd_workspace_size(int B, int T, int D, int N, int packed) {
  if (B <= 0 || T <= 0 || D <= 0 || !ns_ok(N)) return 0;
  return gla::scan_fwd_workspace(B, packed ? (long long)T : (long long)B * T, D, N, packed != 0);
}

gla_status gla_scan_fwd(const void* u, int64_t u_stride, const void* dt, int64_t dt_stride,
                        const float* a, const void* b, int64_t b_stride, const void* c,
                        int64_t c_stride, const float* skip, const void* z, int64_t z_stride,
                        const float* dt_bias, const float* init_state, void* out,
                        float* final_state, const int32_t* cu_seqlens, int B, int T, int D, int N,
                        void* workspace, size_t workspace_bytes, gla_stream_t stream,
                        unsigned flags) {
  if ((flags & ~kScanFlags) != 0u || B < 0 || T < 0 || D < 0) return GLA_ERR_INVALID_ARG;
  if (!ns_ok(N) || !channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (B == 0 || D == 0) return GLA_OK;
  gla::ScanArgs s{};
  const gla_status bad = scan_args(u, u_stride, dt, dt_stride, a, b, b_stride, c, c_stride, skip,
                                   z, z_stride, dt_bias, init_state, cu_seqlens, B, T, D, N,
                                   flags, &s);
  if (bad != GLA_OK) return bad;
  const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
  const long long esz = s.fp32_io ? 4 : 2, osz = s.fp32_out ? 4 : 2;
  if (rows > 0 && !out) return GLA_ERR_INVALID_ARG;
  if (rows == 0 && !final_state) return GLA_OK;
  if (!aligned(out, 16) || !aligned(final_state, 16) || !aligned(workspace, 256))
    return GLA_ERR_MISALIGNED;
  const size_t need = rows > 0 ? gla::scan_fwd_workspace(B, rows, D, N, cu_seqlens) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GLA_ERR_INVALID_ARG;
  const size_t st = (size_t)((long long)B * D * N) * 4;
  const Range in[] = {GLA_SCAN_INPUTS(s, rows, esz),
                      {init_state == final_state ? nullptr : init_state, st}};
  const Range outs[] = {{out, (size_t)(rows * D * osz)}, {final_state, st}, {workspace, need}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  s.status = gla::device_status_word(&err);
  if (!s.status) return finish(err);
  s.out = out; s.final_state = final_state;
  return finish(gla::launch_scan_fwd(s, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gla_scan_bwd_workspace_size(int B, int T, int D, int N, int packed) {
  if (B <= 0 || T < 0 || D <= 0 || !ns_ok(N)) return 0;
  return gla::scan_bwd_workspace(B, packed ? (long long)T : (long long)B * T, D, N);
}

gla_status gla_scan_bwd(const void* u, int64_t u_stride, const void* dt, int64_t dt_stride,
                        const float* a, const void* b, int64_t b_stride, const void* c,
                        int64_t c_stride, const float* skip, const void* z, int64_t z_stride,
                        const float* dt_bias, const float* init_state, const void* d_out,
                        const float* d_final_state, void* du, void* ddt, float* da, void* db,
                        void* dc, float* dskip, void* dz, float* ddt_bias, float* d_init_state,
                        const int32_t* cu_seqlens, int B, int T, int D, int N, void* workspace,
                        size_t workspace_bytes, gla_stream_t stream, unsigned flags) {
  if ((flags & ~kScanFlags) != 0u || B < 0 || T < 0 || D < 0) return GLA_ERR_INVALID_ARG;
  if (!ns_ok(N) || !channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (D == 0) return GLA_OK;
  gla::ScanBwdArgs g{};
  const gla_status bad = scan_args(u, u_stride, dt, dt_stride, a, b, b_stride, c, c_stride, skip,
                                   z, z_stride, dt_bias, init_state, cu_seqlens, B, T, D, N,
                                   flags, &g.f);
  if (bad != GLA_OK) return bad;
  const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
  const long long esz = g.f.fp32_io ? 4 : 2, osz = g.f.fp32_out ? 4 : 2;
  if (!da || (rows > 0 && (B == 0 || !d_out || !du || !ddt || !db || !dc || (z && !dz))) || (!z && dz) ||
      (!skip && dskip) || (!dt_bias && ddt_bias))
    return GLA_ERR_INVALID_ARG;
  if (!aligned(d_out, 16) || !aligned(d_final_state, 16) || !aligned(du, 16) ||
      !aligned(ddt, 16) || !aligned(da, 16) || !aligned(db, 16) || !aligned(dc, 16) ||
      !aligned(dz, 16) || !aligned(dskip, 4) || !aligned(ddt_bias, 4) ||
      !aligned(d_init_state, 16) || !aligned(workspace, 256))
    return GLA_ERR_MISALIGNED;
  const size_t need = gla::scan_bwd_workspace(B, rows, D, N);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GLA_ERR_INVALID_ARG;
  const size_t st = (size_t)((long long)B * D * N) * 4;
  const Range in[] = {GLA_SCAN_INPUTS(g.f, rows, esz),
                      {init_state, st},
                      {d_out, (size_t)(rows * D * esz)},
                      {d_final_state, st}};
  const size_t wide = (size_t)(rows * D * osz), narrow = (size_t)(rows * N * osz);
  const Range outs[] = {{du, wide}, {ddt, wide}, {dz, wide}, {db, narrow}, {dc, narrow},
                        {da, (size_t)D * N * 4}, {dskip, (size_t)D * 4},
                        {ddt_bias, (size_t)D * 4}, {d_init_state, st}, {workspace, need}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  g.f.status = gla::device_status_word(&err);
  if (!g.f.status) return finish(err);
  g.d_out = d_out; g.d_final_state = d_final_state; g.du = du; g.ddt = ddt; g.db = db;
  g.dc = dc; g.dz = dz; g.da = da; g.dskip = dskip; g.ddt_bias = ddt_bias;
  g.d_init_state = d_init_state;
  return finish(gla::launch_scan_bwd(g, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

gla_status gla_scan_step(const void* u, int64_t u_stride, const void* dt, int64_t dt_stride,
                         const float* a, const void* b, int64_t b_stride, const void* c,
                         int64_t c_stride, const float* skip, const void* z, int64_t z_stride,
                         const float* dt_bias, float* state, int num_slots, const int32_t* slots,
                         const int32_t* out_slots, void* out, int rows, int D, int N,
                         gla_stream_t stream, unsigned flags) {
  if ((flags & ~kScanFlags) != 0u || rows < 0 || D < 0 || num_slots < 0 ||
      (!slots && (num_slots != 0 || out_slots)))
    return GLA_ERR_INVALID_ARG;
  if (!ns_ok(N) || !channels_ok(D)) return GLA_ERR_UNSUPPORTED;
  if (rows == 0 || D == 0) return GLA_OK;
  gla::ScanArgs s{};
  const gla_status bad = scan_args(u, u_stride, dt, dt_stride, a, b, b_stride, c, c_stride, skip,
                                   z, z_stride, dt_bias, nullptr, nullptr, rows, 1, D, N, flags,
                                   &s);
  if (bad != GLA_OK) return bad;
  const long long esz = s.fp32_io ? 4 : 2, osz = s.fp32_out ? 4 : 2;
  const long long pages = slots ? num_slots : rows;
  if (pages * D * N > kMaxElems || rows > 65535 * 1024 || (!state && pages > 0) || !out)
    return GLA_ERR_INVALID_ARG;
  if (!aligned(state, 16) || !aligned(out, 16) || !aligned(slots, 4) || !aligned(out_slots, 4))
    return GLA_ERR_MISALIGNED;
  const Range in[] = {GLA_SCAN_INPUTS(s, rows, esz),
                      {slots, (size_t)rows * 4},
                      {out_slots, (size_t)rows * 4}};
  const Range outs[] = {{out, (size_t)((long long)rows * D * osz)},
                        {state, (size_t)(pages * D * N) * 4}};
  if (!disjoint(in, outs)) return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  gla::ScanStepArgs t{};
  t.status = gla::device_status_word(&err);
  if (!t.status) return finish(err);
  t.u = u; t.dt = dt; t.b = b; t.c = c; t.z = z;
  t.u_stride = u_stride; t.dt_stride = dt_stride; t.b_stride = b_stride; t.c_stride = c_stride;
  t.z_stride = z_stride; t.a = a; t.skip = skip; t.dt_bias = dt_bias; t.state = state;
  t.num_slots = num_slots; t.slots = slots; t.out_slots = out_slots; t.out = out;
  t.N = rows; t.D = D; t.NS = N; t.softplus = s.softplus; t.fp32_io = s.fp32_io;
  t.fp32_out = s.fp32_out;
  return finish(gla::launch_scan_step(t, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// The pools of a page operator: pages of a multiple of 16 bytes, 16-byte
// aligned, apart from one another and from the tables.
gla_status check_pools(const gla_page_pool* pools, int count, int num_pages, const Range* tables,
                       int num_tables) {
  if (count < 0 || num_pages < 0 || (count > 0 && !pools)) return GLA_ERR_INVALID_ARG;
  if (num_pages > GLA_MAX_PAGES) return GLA_ERR_UNSUPPORTED;
  for (int i = 0; i < count; ++i) {
    if (!pools[i].base || pools[i].page_bytes <= 0) return GLA_ERR_INVALID_ARG;
    if (!aligned(pools[i].base, 16) || pools[i].page_bytes % 16 != 0) return GLA_ERR_MISALIGNED;
    if (pools[i].page_bytes > (1ll << 32)) return GLA_ERR_UNSUPPORTED;
    const Range p{pools[i].base, (size_t)(pools[i].page_bytes * num_pages)};
    for (int j = 0; j < i; ++j)
      if (overlap(p, {pools[j].base, (size_t)(pools[j].page_bytes * num_pages)}))
        return GLA_ERR_INVALID_ARG;
    for (int t = 0; t < num_tables; ++t)
      if (overlap(p, tables[t])) return GLA_ERR_INVALID_ARG;
  }
  for (int t = 0; t < num_tables; ++t)
    if (!aligned(tables[t].p, 4)) return GLA_ERR_MISALIGNED;
  return GLA_OK;
}

static_assert(sizeof(gla_page_pool) == sizeof(gla::PagePool), "one layout");
const gla::PagePool* as_pools(const gla_page_pool* p) {
  return reinterpret_cast<const gla::PagePool*>(p);
}

// two tables that must be apart, or the same one exactly
bool apart_or_same(const Range& a, const Range& b) { return a.p == b.p || !overlap(a, b); }

}  // namespace

extern "C" {

gla_status gla_pages_copy(const gla_page_pool* pools, int num_pools, int num_pages,
                          const int32_t* src, const int32_t* dst, int32_t* copied, int n,
                          gla_stream_t stream) {
  if (n < 0) return GLA_ERR_INVALID_ARG;
  const size_t nb = (size_t)n * 4;
  const Range t[] = {{src, nb}, {dst, nb}, {copied, nb}};
  const gla_status bad = check_pools(pools, num_pools, num_pages, t, 3);
  if (bad != GLA_OK) return bad;
  if (n == 0) return GLA_OK;
  if (!src || !dst || !copied || overlap(t[2], t[0]) || overlap(t[2], t[1]))
    return GLA_ERR_INVALID_ARG;
  cudaError_t err;
  unsigned* status = gla::device_status_word(&err);
  if (!status) return finish(err);
  return finish(gla::launch_pages_copy(as_pools(pools), num_pools, num_pages, src, dst, copied, n,
                                       status, reinterpret_cast<cudaStream_t>(stream)));
}

gla_status gla_pages_fork(const gla_page_pool* pools, int num_pools, int num_pages,
                          const int32_t* used, int32_t* used_out, const int32_t* parents,
                          int32_t* children, int n, gla_stream_t stream) {
  if (n < 0) return GLA_ERR_INVALID_ARG;
  const size_t nb = (size_t)n * 4, ub = (size_t)(num_pages > 0 ? num_pages : 0) * 4;
  const Range t[] = {{used, ub}, {used_out, ub}, {parents, nb}, {children, nb}};
  const gla_status bad = check_pools(pools, num_pools, num_pages, t, 4);
  if (bad != GLA_OK) return bad;
  if (num_pages > 0 && (!used || !used_out)) return GLA_ERR_INVALID_ARG;
  if (n > 0 && (!parents || !children)) return GLA_ERR_INVALID_ARG;
  if (!apart_or_same(t[0], t[1]) || overlap(t[3], t[0]) || overlap(t[3], t[1]) ||
      overlap(t[3], t[2]) || overlap(t[2], t[1]))
    return GLA_ERR_INVALID_ARG;
  if (n == 0 && (num_pages == 0 || used == used_out)) return GLA_OK;
  cudaError_t err;
  unsigned* status = gla::device_status_word(&err);
  if (!status) return finish(err);
  return finish(gla::launch_pages_fork(as_pools(pools), num_pools, num_pages, used, used_out,
                                       parents, children, n, status,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

gla_status gla_pages_compact(const gla_page_pool* pools, int num_pools, int num_pages,
                             const int32_t* used, int32_t* used_out, const int32_t* slots,
                             int32_t* slots_out, int n, int32_t* forward, gla_stream_t stream) {
  if (n < 0) return GLA_ERR_INVALID_ARG;
  const size_t nb = (size_t)n * 4, ub = (size_t)(num_pages > 0 ? num_pages : 0) * 4;
  const Range t[] = {{used, ub}, {used_out, ub}, {slots, nb}, {slots_out, nb}, {forward, ub}};
  const gla_status bad = check_pools(pools, num_pools, num_pages, t, 5);
  if (bad != GLA_OK) return bad;
  if (num_pages > 0 && (!used || !used_out || !forward)) return GLA_ERR_INVALID_ARG;
  if (n > 0 && (!slots || !slots_out)) return GLA_ERR_INVALID_ARG;
  if (!apart_or_same(t[0], t[1]) || !apart_or_same(t[2], t[3])) return GLA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    for (int j = 2; j < 5; ++j)
      if (overlap(t[i], t[j])) return GLA_ERR_INVALID_ARG;
  if (overlap(t[4], t[2]) || overlap(t[4], t[3])) return GLA_ERR_INVALID_ARG;
  if (num_pages == 0 && n == 0) return GLA_OK;
  cudaError_t err;
  unsigned* status = gla::device_status_word(&err);
  if (!status) return finish(err);
  return finish(gla::launch_pages_compact(as_pools(pools), num_pools, num_pages, used, used_out,
                                          slots, slots_out, n, forward, status,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

gla_status gla_pages_free(const int32_t* used, int32_t* used_out, int num_pages,
                          const int32_t* slots, int n, gla_stream_t stream) {
  if (n < 0) return GLA_ERR_INVALID_ARG;
  const size_t nb = (size_t)n * 4, ub = (size_t)(num_pages > 0 ? num_pages : 0) * 4;
  const Range t[] = {{used, ub}, {used_out, ub}, {slots, nb}};
  const gla_status bad = check_pools(nullptr, 0, num_pages, t, 3);
  if (bad != GLA_OK) return bad;
  if ((num_pages > 0 && (!used || !used_out)) || (n > 0 && !slots)) return GLA_ERR_INVALID_ARG;
  if (!apart_or_same(t[0], t[1]) || overlap(t[2], t[1])) return GLA_ERR_INVALID_ARG;
  if (n == 0 && (num_pages == 0 || used == used_out)) return GLA_OK;
  cudaError_t err;
  unsigned* status = gla::device_status_word(&err);
  if (!status) return finish(err);
  return finish(gla::launch_pages_free(num_pages, used, used_out, slots, n, status,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
