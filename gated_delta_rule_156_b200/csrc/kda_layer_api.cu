// C-ABI boundary of the layer operators (include/kda_layer.h): argument
// validation, workspace, dispatch.  Every argument error is found here, on
// the host, before anything launches.
#include "../../include/kda_layer.h"

#include <math.h>
#include <stdint.h>

#include "kda_layer_internal.h"
#include "kda_ssm.cuh"

namespace {

constexpr int kMaxChannels = 1 << 20;

kda_status done(cudaError_t e) {
  if (e == cudaSuccess) return KDA_OK;
  kda::api_record_cuda_error(e);
  return KDA_ERR_CUDA;
}

// Runs `launch` with stream-ordered workspace.
template <typename F>
kda_status with_workspace(size_t bytes, cudaStream_t stream, F launch) {
  void* ws = nullptr;
  cudaError_t e = kda::api_take_workspace(bytes, stream, &ws);
  if (e == cudaSuccess) e = launch(ws);
  if (ws) {
    const cudaError_t f = cudaFreeAsync(ws, stream);
    if (e == cudaSuccess) e = f;
  }
  return done(e);
}

// The memory of one argument.
struct Span {
  const void* p;
  size_t bytes;
  size_t align;
};
// `tokens` slices of `width` elements, `stride` elements apart.
Span rows(const void* p, int64_t tokens, int64_t stride, int64_t width, size_t e) {
  return Span{p, tokens > 0 ? (size_t)((tokens - 1) * stride + width) * e : 0, e};
}
Span flat(const void* p, int64_t n, size_t e) { return Span{p, (size_t)n * e, e}; }

bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// Alignment of everything, no output over an input or another output.
kda_status check_memory(const Span* in, int n_in, const Span* out, int n_out) {
  for (int i = 0; i < n_in; ++i)
    if (in[i].p && (uintptr_t)in[i].p % in[i].align) return KDA_ERR_MISALIGNED;
  for (int i = 0; i < n_out; ++i)
    if (out[i].p && (uintptr_t)out[i].p % out[i].align) return KDA_ERR_MISALIGNED;
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j])) return KDA_ERR_INVALID_ARG;
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(out[i], out[j])) return KDA_ERR_INVALID_ARG;
  }
  return KDA_OK;
}

size_t elem(kda_dtype t) { return t == KDA_BF16 ? 2 : 4; }
bool dtype_ok(int t) { return t == KDA_BF16 || t == KDA_F32; }

// A token stride: 0 is dense; tokens must not overlap.  Below 2^30 elements, so
// that 2^31 tokens of them are counted in 64 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 30;
bool stride_of(int64_t given, int64_t width, int64_t* s) {
  *s = given ? given : width;
  return *s >= width && *s <= kMaxStride;
}

// B, T, n_seqs of a dense or packed batch.
kda_status check_batch(int B, int T, int n_given, bool packed, int* n_seqs, int64_t* tokens) {
  if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
  *n_seqs = B;
  if (packed) {
    if (B != 1 || n_given < 1) return KDA_ERR_INVALID_ARG;
    *n_seqs = n_given;
  }
  *tokens = (int64_t)B * T;
  return *tokens > INT32_MAX - 4096 ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// ---- short convolution ---------------------------------------------------

kda_status conv_args(const kda_conv_shape* s, bool packed, kda::ConvArgs* a) {
  if (!s) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_batch(s->B, s->T, s->n_seqs, packed, &a->n_seqs, &a->tokens);
  if (st != KDA_OK) return st;
  if (s->D < 1 || !dtype_ok(s->io_dtype)) return KDA_ERR_INVALID_ARG;
  if (s->activation != KDA_ACT_NONE && s->activation != KDA_ACT_SILU)
    return KDA_ERR_INVALID_ARG;
  if (!stride_of(s->x_stride, s->D, &a->x_stride)) return KDA_ERR_INVALID_ARG;
  if (s->W < 2 || s->W > 4 || s->D > kMaxChannels || a->n_seqs > INT32_MAX / 8)
    return KDA_ERR_UNSUPPORTED;
  a->T = s->T;
  a->D = s->D;
  a->W = s->W;
  a->act = s->activation;
  a->bf16 = s->io_dtype == KDA_BF16;
  return KDA_OK;
}

// ---- selective scan ------------------------------------------------------

kda_status ssm_args(const kda_ssm_shape* s, bool packed, kda::SsmArgs* a) {
  if (!s) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_batch(s->B, s->T, s->n_seqs, packed, &a->n_seqs, &a->tokens);
  if (st != KDA_OK) return st;
  if (s->D < 1 || s->S < 1 || s->G < 1 || s->D % s->G || !dtype_ok(s->io_dtype))
    return KDA_ERR_INVALID_ARG;
  if (s->S > 128 || s->D > kMaxChannels) return KDA_ERR_UNSUPPORTED;
  a->T = s->T;
  a->D = s->D;
  a->S = s->S;
  a->G = s->G;
  a->bf16 = s->io_dtype == KDA_BF16;
  a->softplus = s->softplus != 0;
  a->b_group = s->b_group_stride ? s->b_group_stride : s->S;
  a->c_group = s->c_group_stride ? s->c_group_stride : s->S;
  if (a->b_group < s->S || a->c_group < s->S || a->b_group > kMaxStride ||
      a->c_group > kMaxStride)
    return KDA_ERR_INVALID_ARG;
  if (!stride_of(s->u_stride, s->D, &a->u_stride) ||
      !stride_of(s->delta_stride, s->D, &a->delta_stride) ||
      !stride_of(s->z_stride, s->D, &a->z_stride))
    return KDA_ERR_INVALID_ARG;
  // a token's groups: the last one starts at (G - 1) group strides
  const int64_t bw = (s->G - 1) * a->b_group + s->S, cw = (s->G - 1) * a->c_group + s->S;
  a->b_stride = s->b_stride ? s->b_stride : (int64_t)s->G * a->b_group;
  a->c_stride = s->c_stride ? s->c_stride : (int64_t)s->G * a->c_group;
  if (a->b_stride < bw || a->c_stride < cw || a->b_stride > kMaxStride ||
      a->c_stride > kMaxStride)
    return KDA_ERR_INVALID_ARG;
  // CTAs (of segments of 128 tokens at the least, where a scan is split) and
  // the backward's sums are counted in 31 bits
  const int ch = kda::kSsmThreads / kda::ssm_lanes(s->S);
  if ((int64_t)kda::ssm_blocks(*a, ch) * (a->n_seqs + a->tokens / 128 + 1) > INT32_MAX ||
      a->tokens * s->G * s->S > ((int64_t)1 << 38) ||
      (int64_t)a->n_seqs * s->D > ((int64_t)1 << 33))
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

struct SsmSpans {
  Span u, delta, B, C, z, A, skip, bias, h0, cu;
};
SsmSpans ssm_spans(const kda::SsmArgs& a) {
  const size_t e = a.bf16 ? 2 : 4;
  const int64_t state = (int64_t)a.n_seqs * a.D * a.S;
  return SsmSpans{rows(a.u, a.tokens, a.u_stride, a.D, e),
                  rows(a.delta, a.tokens, a.delta_stride, a.D, e),
                  rows(a.B, a.tokens, a.b_stride, (a.G - 1) * a.b_group + a.S, e),
                  rows(a.C, a.tokens, a.c_stride, (a.G - 1) * a.c_group + a.S, e),
                  rows(a.z, a.tokens, a.z_stride, a.D, e),
                  flat(a.A, (int64_t)a.D * a.S, 4),
                  flat(a.skip, a.D, 4),
                  flat(a.bias, a.D, 4),
                  flat(a.h0, state, 4),
                  flat(a.cu, a.cu ? (int64_t)a.n_seqs + 1 : 0, 4)};
}

// ---- block norm ------------------------------------------------------------

kda_status norm_args(const kda_norm_shape* s, kda::NormArgs* a) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->tokens < 0 || s->heads < 1 || s->width < 1 || !dtype_ok(s->io_dtype) ||
      !dtype_ok(s->residual_dtype))
    return KDA_ERR_INVALID_ARG;
  if (s->gate_act < KDA_ACT_NONE || s->gate_act > KDA_ACT_SIGMOID) return KDA_ERR_INVALID_ARG;
  if (!(s->eps >= 0.f) || isinf(s->eps)) return KDA_ERR_INVALID_ARG;
  if (s->width > 16384 || s->heads > 65535) return KDA_ERR_UNSUPPORTED;
  if (s->io_dtype == KDA_F32 && s->residual_dtype != KDA_F32) return KDA_ERR_UNSUPPORTED;
  const int64_t w = (int64_t)s->heads * s->width;
  if (s->tokens > INT32_MAX || w > kMaxStride) return KDA_ERR_UNSUPPORTED;
  if (!stride_of(s->x_stride, w, &a->x_stride) || !stride_of(s->gate_stride, w, &a->gate_stride))
    return KDA_ERR_INVALID_ARG;
  a->tokens = s->tokens;
  a->heads = s->heads;
  a->width = s->width;
  a->act = s->gate_act;
  a->gate_first = s->gate_first != 0;
  a->eps = s->eps;
  a->bf16 = s->io_dtype == KDA_BF16;
  a->res_bf16 = s->residual_dtype == KDA_BF16;
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_short_conv_fwd(const kda_conv_shape* shape, const void* x, const float* weight,
                              const float* bias, const void* initial_state,
                              const int32_t* cu_seqlens, void* out, void* final_state,
                              cudaStream_t stream) {
  kda::ConvArgs a{};
  kda_status st = conv_args(shape, cu_seqlens != nullptr, &a);
  if (st != KDA_OK) return st;
  if (!weight || (a.tokens && (!x || !out))) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(shape->io_dtype);
  const int64_t state = (int64_t)a.n_seqs * (a.W - 1) * a.D;
  const Span in[] = {rows(x, a.tokens, a.x_stride, a.D, e), flat(weight, (int64_t)a.D * a.W, 4),
                     flat(bias, a.D, 4), flat(initial_state, state, e),
                     flat(cu_seqlens, (int64_t)a.n_seqs + 1, 4)};
  const Span outs[] = {flat(out, a.tokens * a.D, e), flat(final_state, state, e)};
  if ((st = check_memory(in, 5, outs, 2)) != KDA_OK) return st;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.past = initial_state;
  a.cu = cu_seqlens;
  a.out = out;
  a.final_state = final_state;
  return done(kda::launch_conv_fwd(a, stream));
}

kda_status kda_short_conv_bwd(const kda_conv_shape* shape, const void* x, const float* weight,
                              const float* bias, const void* initial_state,
                              const int32_t* cu_seqlens, const void* d_out,
                              const void* d_final_state, void* dx, float* d_weight,
                              float* d_bias, void* d_initial_state, cudaStream_t stream) {
  kda::ConvArgs a{};
  kda_status st = conv_args(shape, cu_seqlens != nullptr, &a);
  if (st != KDA_OK) return st;
  if (!weight || !d_weight || (a.tokens && (!x || !d_out || !dx))) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(shape->io_dtype);
  const int64_t state = (int64_t)a.n_seqs * (a.W - 1) * a.D;
  const Span in[] = {rows(x, a.tokens, a.x_stride, a.D, e),
                     flat(weight, (int64_t)a.D * a.W, 4),
                     flat(bias, a.D, 4),
                     flat(initial_state, state, e),
                     flat(cu_seqlens, (int64_t)a.n_seqs + 1, 4),
                     flat(d_out, a.tokens * a.D, e),
                     flat(d_final_state, state, e)};
  const Span outs[] = {flat(dx, a.tokens * a.D, e), flat(d_weight, (int64_t)a.D * a.W, 4),
                       flat(d_bias, a.D, 4), flat(d_initial_state, state, e)};
  if ((st = check_memory(in, 7, outs, 4)) != KDA_OK) return st;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.past = initial_state;
  a.cu = cu_seqlens;
  a.d_out = d_out;
  a.d_final = d_final_state;
  a.dx = dx;
  a.dw = d_weight;
  a.db = d_bias;
  a.d_past = d_initial_state;
  return with_workspace(kda::conv_bwd_workspace_bytes(a), stream,
                        [&](void* ws) { return kda::launch_conv_bwd(a, ws, stream); });
}

kda_status kda_short_conv_step(const kda_conv_shape* shape, const void* x, const float* weight,
                               const float* bias, void* state_inout, void* out,
                               cudaStream_t stream) {
  kda::ConvArgs a{};
  kda_status st = conv_args(shape, false, &a);
  if (st != KDA_OK) return st;
  if (!weight || (a.n_seqs && !state_inout) || (a.tokens && (!x || !out)))
    return KDA_ERR_INVALID_ARG;
  const size_t e = elem(shape->io_dtype);
  const Span in[] = {rows(x, a.tokens, a.x_stride, a.D, e), flat(weight, (int64_t)a.D * a.W, 4),
                     flat(bias, a.D, 4)};
  const Span outs[] = {flat(out, a.tokens * a.D, e),
                       flat(state_inout, (int64_t)a.n_seqs * (a.W - 1) * a.D, e)};
  if ((st = check_memory(in, 3, outs, 2)) != KDA_OK) return st;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.out = out;
  a.final_state = state_inout;
  return done(kda::launch_conv_step(a, stream));
}

kda_status kda_ssm_scan_fwd(const kda_ssm_shape* shape, const void* u, const void* delta,
                            const float* A, const void* Bm, const void* Cm, const float* skip,
                            const void* z, const float* delta_bias, const float* initial_state,
                            const int32_t* cu_seqlens, void* out, float* final_state,
                            cudaStream_t stream) {
  kda::SsmArgs a{};
  kda_status st = ssm_args(shape, cu_seqlens != nullptr, &a);
  if (st != KDA_OK) return st;
  if (!A || (a.tokens && (!u || !delta || !Bm || !Cm || !out))) return KDA_ERR_INVALID_ARG;
  a.u = u;
  a.delta = delta;
  a.A = A;
  a.B = Bm;
  a.C = Cm;
  a.skip = skip;
  a.z = z;
  a.bias = delta_bias;
  a.h0 = initial_state;
  a.cu = cu_seqlens;
  a.out = out;
  a.h_out = final_state;
  const SsmSpans s = ssm_spans(a);
  const Span so = flat(out, a.tokens * a.D, elem(shape->io_dtype)),
             sf = flat(final_state, (int64_t)a.n_seqs * a.D * a.S, 4);
  const Span in[] = {s.u, s.delta, s.B, s.C, s.z, s.A, s.skip, s.bias, s.cu, s.h0};
  // the final state may coincide exactly with the initial state
  const bool same = final_state && final_state == initial_state;
  const Span outs[] = {so, sf};
  if ((st = check_memory(in, same ? 9 : 10, outs, 2)) != KDA_OK) return st;
  const int sms = kda::sm_count();
  return with_workspace(kda::ssm_fwd_workspace_bytes(a, sms), stream,
                        [&](void* ws) { return kda::launch_ssm_fwd(a, ws, sms, stream); });
}

static kda_status ssm_bwd_args(const kda_ssm_shape* shape, bool packed, kda::SsmBwdArgs* b) {
  return ssm_args(shape, packed, &b->f);
}

kda_status kda_ssm_scan_bwd(const kda_ssm_shape* shape, const void* u, const void* delta,
                            const float* A, const void* Bm, const void* Cm, const float* skip,
                            const void* z, const float* delta_bias, const float* initial_state,
                            const int32_t* cu_seqlens, const void* d_out,
                            const float* d_final_state, void* du, void* ddelta, float* dA,
                            void* dBm, void* dCm, float* d_skip, void* dz, float* d_delta_bias,
                            float* d_initial_state, cudaStream_t stream) {
  kda::SsmBwdArgs b{};
  kda_status st = ssm_bwd_args(shape, cu_seqlens != nullptr, &b);
  if (st != KDA_OK) return st;
  kda::SsmArgs& a = b.f;
  if (!A || !dA || (a.tokens && (!u || !delta || !Bm || !Cm || !d_out || !du || !ddelta ||
                                 !dBm || !dCm)))
    return KDA_ERR_INVALID_ARG;
  // a gradient is asked for exactly with its input (z has values to write)
  if ((d_skip && !skip) || (d_delta_bias && !delta_bias) || (dz && !z) ||
      (a.tokens && z && !dz))
    return KDA_ERR_INVALID_ARG;
  a.u = u;
  a.delta = delta;
  a.A = A;
  a.B = Bm;
  a.C = Cm;
  a.skip = skip;
  a.z = z;
  a.bias = delta_bias;
  a.h0 = initial_state;
  a.cu = cu_seqlens;
  b.d_out = d_out;
  b.d_final = d_final_state;
  b.du = du;
  b.ddelta = ddelta;
  b.dA = dA;
  b.dB = dBm;
  b.dC = dCm;
  b.dskip = d_skip;
  b.dz = dz;
  b.dbias = d_delta_bias;
  b.dh0 = d_initial_state;
  const size_t e = elem(shape->io_dtype);
  const SsmSpans s = ssm_spans(a);
  const int64_t state = (int64_t)a.n_seqs * a.D * a.S, bc = a.tokens * a.G * a.S;
  const Span in[] = {s.u, s.delta, s.B, s.C, s.z, s.A, s.skip, s.bias, s.cu, s.h0,
                     flat(d_out, a.tokens * a.D, e), flat(d_final_state, state, 4)};
  const Span outs[] = {flat(du, a.tokens * a.D, e), flat(ddelta, a.tokens * a.D, e),
                       flat(dA, (int64_t)a.D * a.S, 4), flat(dBm, bc, e), flat(dCm, bc, e),
                       flat(d_skip, a.D, 4), flat(dz, a.tokens * a.D, e),
                       flat(d_delta_bias, a.D, 4), flat(d_initial_state, state, 4)};
  if ((st = check_memory(in, 12, outs, 9)) != KDA_OK) return st;
  const int sms = kda::sm_count();
  return with_workspace(kda::ssm_bwd_workspace_bytes(b, sms), stream,
                        [&](void* ws) { return kda::launch_ssm_bwd(b, ws, sms, stream); });
}

kda_status kda_ssm_scan_bwd_plan(const kda_ssm_shape* shape, int packed, int* kernels,
                                 size_t* workspace_bytes) {
  kda::SsmBwdArgs b{};
  const kda_status st = ssm_bwd_args(shape, packed != 0, &b);
  if (st != KDA_OK) return st;
  static const int32_t tag = 0;  // only tells the planner the layout
  b.f.cu = packed ? &tag : nullptr;
  const int sms = kda::sm_count();
  if (kernels) *kernels = kda::ssm_bwd_kernel_count(b, sms);
  if (workspace_bytes) *workspace_bytes = kda::ssm_bwd_workspace_bytes(b, sms);
  return KDA_OK;
}

kda_status kda_ssm_step(const kda_ssm_shape* shape, const void* u, const void* delta,
                        const float* A, const void* Bm, const void* Cm, const float* skip,
                        const void* z, const float* delta_bias, float* state_inout, void* out,
                        cudaStream_t stream) {
  kda::SsmArgs a{};
  kda_status st = ssm_args(shape, false, &a);
  if (st != KDA_OK) return st;
  if (!A || (a.n_seqs && !state_inout) ||
      (a.tokens && (!u || !delta || !Bm || !Cm || !out)))
    return KDA_ERR_INVALID_ARG;
  a.u = u;
  a.delta = delta;
  a.A = A;
  a.B = Bm;
  a.C = Cm;
  a.skip = skip;
  a.z = z;
  a.bias = delta_bias;
  a.out = out;
  a.h_out = state_inout;
  const SsmSpans s = ssm_spans(a);
  const Span in[] = {s.u, s.delta, s.B, s.C, s.z, s.A, s.skip, s.bias};
  const Span outs[] = {flat(out, a.tokens * a.D, elem(shape->io_dtype)),
                       flat(state_inout, (int64_t)a.n_seqs * a.D * a.S, 4)};
  if ((st = check_memory(in, 8, outs, 2)) != KDA_OK) return st;
  return done(kda::launch_ssm_step(a, stream));
}

kda_status kda_block_norm_fwd(const kda_norm_shape* shape, const void* x,
                              const float* post_weight, const void* gate, const void* residual,
                              const float* scale, const float* pre_weight, void* out,
                              void* normed, cudaStream_t stream) {
  kda::NormArgs a{};
  kda_status st = norm_args(shape, &a);
  if (st != KDA_OK) return st;
  if (a.tokens && (!x || !out || (pre_weight && !normed))) return KDA_ERR_INVALID_ARG;
  if (normed && !pre_weight) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(shape->io_dtype), r = elem(shape->residual_dtype);
  const int64_t w = (int64_t)a.heads * a.width, n = a.tokens * w;
  const Span in[] = {rows(x, a.tokens, a.x_stride, w, e),
                     rows(gate, a.tokens, a.gate_stride, w, e),
                     flat(post_weight, a.width, 4), flat(scale, a.width, 4),
                     flat(pre_weight, a.width, 4), flat(residual, n, r)};
  const Span outs[] = {flat(out, n, r), flat(normed, n, e)};
  // `out` may be the residual itself
  const bool same = residual && out == residual;
  if ((st = check_memory(in, same ? 5 : 6, outs, 2)) != KDA_OK) return st;
  a.x = x;
  a.gate = gate;
  a.residual = residual;
  a.post_weight = post_weight;
  a.scale = scale;
  a.pre_weight = pre_weight;
  a.out = out;
  a.normed = normed;
  return done(kda::launch_norm_fwd(a, stream));
}

kda_status kda_block_norm_bwd(const kda_norm_shape* shape, const void* x,
                              const float* post_weight, const void* gate, const void* residual,
                              const float* scale, const float* pre_weight, const void* d_out,
                              const void* d_normed, void* dx, void* dgate, void* d_residual,
                              float* d_post_weight, float* d_scale, float* d_pre_weight,
                              cudaStream_t stream) {
  kda::NormArgs a{};
  kda_status st = norm_args(shape, &a);
  if (st != KDA_OK) return st;
  if (a.tokens && (!x || !dx || (gate && !dgate))) return KDA_ERR_INVALID_ARG;
  if ((dgate && !gate) || (d_residual && !residual) || (d_post_weight && !post_weight) ||
      (d_scale && !scale) || (d_pre_weight && !pre_weight) || (d_normed && !pre_weight))
    return KDA_ERR_INVALID_ARG;
  const size_t e = elem(shape->io_dtype), r = elem(shape->residual_dtype);
  const int64_t w = (int64_t)a.heads * a.width, n = a.tokens * w;
  const Span in[] = {rows(x, a.tokens, a.x_stride, w, e),
                     rows(gate, a.tokens, a.gate_stride, w, e),
                     flat(post_weight, a.width, 4), flat(scale, a.width, 4),
                     flat(pre_weight, a.width, 4), flat(residual, n, r),
                     flat(d_out, n, r), flat(d_normed, n, e)};
  const Span outs[] = {flat(dx, n, e), flat(dgate, n, e), flat(d_residual, n, r),
                       flat(d_post_weight, a.width, 4), flat(d_scale, a.width, 4),
                       flat(d_pre_weight, a.width, 4)};
  if ((st = check_memory(in, 8, outs, 6)) != KDA_OK) return st;
  a.x = x;
  a.gate = gate;
  a.residual = residual;
  a.post_weight = post_weight;
  a.scale = scale;
  a.pre_weight = pre_weight;
  a.d_out = d_out;
  a.d_normed = d_normed;
  a.dx = dx;
  a.dgate = dgate;
  a.dres = d_residual;
  a.dpost = d_post_weight;
  a.dscale = d_scale;
  a.dpre = d_pre_weight;
  const int sms = kda::sm_count();
  return with_workspace(kda::norm_bwd_workspace_bytes(a, sms), stream,
                        [&](void* ws) { return kda::launch_norm_bwd(a, ws, sms, stream); });
}

}  // extern "C"
