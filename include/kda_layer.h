/*
 * kda_layer.h -- C ABI of the operators around a recurrent layer: the short
 * causal convolution in front of it, the selective state space scan (the
 * diagonal recurrence that stands beside the delta rule of kda.h), and the
 * norms after and before a block fused with its gate, its residual scale and
 * the residual sum.  Part of libkda.so; statuses, streams, workspace and
 * error reporting are those of kda.h:
 *   - all tensor pointers are device memory owned by the caller, calls are
 *     asynchronous on `stream` of the current device, never synchronise the
 *     host and can be captured into a CUDA graph; workspace, where a call
 *     needs one, is stream-ordered;
 *   - argument errors are found on the host before anything is launched.
 *
 * Layouts are token-major and row-major.  Tensors marked "token stride" may
 * be slices of a wider projection output: the elements of one token are
 * consecutive, and consecutive tokens of the flat [B * T] axis are
 * `*_stride` elements apart (0: dense; at most 2^30).  Every tensor must be aligned to its
 * element (KDA_ERR_MISALIGNED otherwise); 16-byte aligned pointers and
 * strides take the wide loads.
 *
 * Packed batches: as in kda.h, cu_seqlens holds n_seqs + 1 int32 offsets
 * into the token axis and B is 1.  It is device memory and not checked on
 * the host; the kernels clamp every offset into [0, T], and results for an
 * array that decreases are unspecified (in bounds).  Sequences may be empty.
 * Tokens before the first offset or behind the last one belong to no
 * sequence: they are not read, and their outputs are left as they were.
 *
 * Inputs keep their non-finite values: a NaN or an infinity reaches the
 * results that depend on it, and no others.
 */
#ifndef KDA_LAYER_H_
#define KDA_LAYER_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KDA_ACT_NONE = 0,   /* identity              */
  KDA_ACT_SILU = 1,   /* x sigmoid(x)          */
  KDA_ACT_SIGMOID = 2 /* 1 / (1 + exp(-x))     */
} kda_act;

/* ---- short causal convolution ------------------------------------------ */

typedef struct {
  int B;              /* sequences (1 with cu_seqlens)                        */
  int T;              /* tokens per sequence, or all packed tokens            */
  int D;              /* channels                                             */
  int W;              /* taps: 2, 3 or 4                                      */
  int n_seqs;         /* packed sequences (used only with cu_seqlens)         */
  kda_dtype io_dtype; /* dtype of x, out, the states and their gradients      */
  int activation;     /* KDA_ACT_NONE or KDA_ACT_SILU                         */
  int64_t x_stride;   /* token stride of x in elements, 0 = D                 */
} kda_conv_shape;

/*
 * kda_short_conv_fwd -- depthwise causal convolution over each sequence:
 *     pre_t = bias + sum_{j < W} weight[:, j] x_{t - (W-1) + j}
 *     out_t = activation(pre_t)
 * where x at the W - 1 places before a sequence is its initial state (or 0).
 *   x             : [B, T, D] io dtype, token stride.
 *   weight, bias  : [D, W] and [D] fp32; bias may be NULL.
 *   initial_state : [N, W-1, D] io dtype, oldest first, or NULL (zeros).
 *   out           : [B, T, D] io dtype, dense.
 *   final_state   : [N, W-1, D] io dtype or NULL: each sequence's last W - 1
 *                   inputs (a shorter sequence keeps the end of its initial
 *                   state).  An exact copy of inputs.
 * Sums are fp32.  No output may overlap an input or the other output.
 */
KDA_API kda_status kda_short_conv_fwd(const kda_conv_shape* shape,
                                      const void* x, const float* weight,
                                      const float* bias,
                                      const void* initial_state,
                                      const int32_t* cu_seqlens, void* out,
                                      void* final_state, cudaStream_t stream);

/*
 * kda_short_conv_bwd -- gradients of sum(d_out * out) + sum(d_final_state *
 * final_state).  d_out [B, T, D] and d_final_state [N, W-1, D] (or NULL) io
 * dtype, dense.  Writes dx [B, T, D] io dtype; d_weight [D, W] and d_bias [D]
 * fp32 (d_bias may be NULL); d_initial_state [N, W-1, D] io dtype or NULL.
 * The weights' sums over tokens are fp32 in a fixed order: repeats are
 * bit-identical.  Stream-ordered workspace of at most (W + 1) D floats for
 * each 64 tokens (512 in large calls).
 */
KDA_API kda_status kda_short_conv_bwd(
    const kda_conv_shape* shape, const void* x, const float* weight,
    const float* bias, const void* initial_state, const int32_t* cu_seqlens,
    const void* d_out, const void* d_final_state, void* dx, float* d_weight,
    float* d_bias, void* d_initial_state, cudaStream_t stream);

/*
 * kda_short_conv_step -- the convolution of T >= 1 new tokens for each of B
 * sequences (one for a decode step), state_inout [B, W-1, D] io dtype updated
 * in place.  No packed form.
 */
KDA_API kda_status kda_short_conv_step(const kda_conv_shape* shape,
                                       const void* x, const float* weight,
                                       const float* bias, void* state_inout,
                                       void* out, cudaStream_t stream);

/* ---- selective state space scan ----------------------------------------- */

typedef struct {
  int B;                  /* sequences (1 with cu_seqlens)                    */
  int T;                  /* tokens per sequence, or all packed tokens        */
  int D;                  /* channels                                         */
  int S;                  /* states per channel, 1 .. 128                     */
  int G;                  /* groups of B and C; divides D                     */
  int n_seqs;             /* packed sequences (used only with cu_seqlens)     */
  kda_dtype io_dtype;     /* dtype of u, delta, z, B, C, out, their gradients */
  int softplus;           /* nonzero: step = softplus(delta + delta_bias)     */
  int64_t u_stride;       /* token strides in elements, 0 = dense             */
  int64_t delta_stride;
  int64_t z_stride;
  int64_t b_stride, b_group_stride; /* of B: between tokens, between groups   */
  int64_t c_stride, c_group_stride; /* of C                                   */
} kda_ssm_shape;

/*
 * kda_ssm_scan_fwd -- per sequence, channel d (of group g) and state n:
 *     step_t = softplus(delta_t + delta_bias)       (or delta_t + delta_bias)
 *     h_t[n] = exp(step_t A[d, n]) h_{t-1}[n] + step_t u_t B_t[g, n]
 *     y_t    = sum_n C_t[g, n] h_t[n] + skip[d] u_t
 *     out_t  = y_t silu(z_t)                        (y_t without z)
 *   u, delta, z : [B, T, D] io dtype, token strides; z may be NULL.
 *   A           : [D, S] fp32, finite, used as given (negative for a decay).
 *   Bm, Cm      : [B, T, G, S] io dtype, token and group strides.
 *   skip, delta_bias : [D] fp32, may be NULL.
 *   initial_state : [N, D, S] fp32, or NULL (zeros).
 *   out         : [B, T, D] io dtype, dense.
 *   final_state : [N, D, S] fp32 or NULL; may equal initial_state.
 * The state and all sums are fp32.  Long sequences that would leave most of
 * the SMs idle are scanned in segments side by side, which are then joined
 * (exactly: the recurrence is linear in the state); that takes stream-ordered
 * workspace of D (S + 1) floats a segment.
 * An infinite state stays infinite while its tokens' decays are above 0 in
 * fp32, split or not (0 times infinity, behind such a decay, may be NaN).
 */
KDA_API kda_status kda_ssm_scan_fwd(
    const kda_ssm_shape* shape, const void* u, const void* delta,
    const float* A, const void* Bm, const void* Cm, const float* skip,
    const void* z, const float* delta_bias, const float* initial_state,
    const int32_t* cu_seqlens, void* out, float* final_state,
    cudaStream_t stream);

/*
 * kda_ssm_scan_bwd -- gradients of sum(d_out * out) + sum(d_final_state *
 * final_state).  d_out [B, T, D] io dtype dense; d_final_state [N, D, S] fp32
 * or NULL.  Writes, all dense: du, ddelta, dz [B, T, D] io dtype (dz only with
 * z); dA [D, S], d_skip [D] (only with skip), d_delta_bias [D] (only with
 * delta_bias) fp32; dBm, dCm [B, T, G, S] io dtype; d_initial_state [N, D, S]
 * fp32 or NULL.  All sums are fp32 in a fixed order: repeats are
 * bit-identical.  The call runs the forward recurrence again and keeps its
 * state at every 8th token in a stream-ordered workspace
 * (kda_ssm_scan_bwd_plan reports its size).
 */
KDA_API kda_status kda_ssm_scan_bwd(
    const kda_ssm_shape* shape, const void* u, const void* delta,
    const float* A, const void* Bm, const void* Cm, const float* skip,
    const void* z, const float* delta_bias, const float* initial_state,
    const int32_t* cu_seqlens, const void* d_out, const float* d_final_state,
    void* du, void* ddelta, float* dA, void* dBm, void* dCm, float* d_skip,
    void* dz, float* d_delta_bias, float* d_initial_state,
    cudaStream_t stream);

/* Kernels a kda_ssm_scan_bwd call of this shape launches and the workspace
 * it allocates on the current device (148 SMs where there is none); no device
 * work.  `packed` selects the cu_seqlens layout. */
KDA_API kda_status kda_ssm_scan_bwd_plan(const kda_ssm_shape* shape,
                                         int packed, int* kernels,
                                         size_t* workspace_bytes);

/*
 * kda_ssm_step -- the scan over T >= 1 new tokens for each of B sequences
 * (one for a decode step), state_inout [B, D, S] fp32 updated in place: each
 * state element is read and written once per call.  No packed form.
 */
KDA_API kda_status kda_ssm_step(const kda_ssm_shape* shape, const void* u,
                                const void* delta, const float* A,
                                const void* Bm, const void* Cm,
                                const float* skip, const void* z,
                                const float* delta_bias, float* state_inout,
                                void* out, cudaStream_t stream);

/* ---- norms at a block's boundary ----------------------------------------- */

typedef struct {
  int64_t tokens;           /* rows / heads                                   */
  int heads;                /* rows per token (1: the norm spans the token)   */
  int width;                /* elements per row, 1 .. 16384                   */
  kda_dtype io_dtype;       /* dtype of x, gate, normed and their gradients   */
  kda_dtype residual_dtype; /* dtype of residual and out: io_dtype or KDA_F32 */
  int gate_act;             /* a kda_act, applied to the gate                 */
  int gate_first;           /* nonzero: gate before the norm                  */
  float eps;                /* >= 0                                           */
  int64_t x_stride;         /* token strides in elements, 0 = heads * width   */
  int64_t gate_stride;
} kda_norm_shape;

/*
 * kda_block_norm_fwd -- per row of `width` elements, with
 * rms(v) = v / sqrt(mean(v^2) + eps):
 *     h      = x                       (x act(gate) with gate_first)
 *     p      = rms(h) post_weight      (h without post_weight)
 *     p      = p act(gate)             (unless gate_first)
 *     out    = residual + scale p      (without residual: scale p)
 *     normed = rms(out) pre_weight     (only with pre_weight)
 * `normed` is formed from the fp32 `out`, before its rounding.
 *   x, gate     : [tokens, heads, width] io dtype, token strides; gate may be
 *                 NULL.
 *   post_weight, scale, pre_weight : [width] fp32, each may be NULL.
 *   residual    : [tokens, heads, width] residual dtype, dense, or NULL (then
 *                 residual_dtype is the dtype of out).
 *   out         : as residual; may be the residual itself (in place).
 *   normed      : [tokens, heads, width] io dtype, dense; NULL without
 *                 pre_weight.
 */
KDA_API kda_status kda_block_norm_fwd(
    const kda_norm_shape* shape, const void* x, const float* post_weight,
    const void* gate, const void* residual, const float* scale,
    const float* pre_weight, void* out, void* normed, cudaStream_t stream);

/*
 * kda_block_norm_bwd -- gradients of sum(d_out * out) + sum(d_normed *
 * normed); the rows are formed again from x, gate and residual.  d_out
 * (residual dtype) and d_normed (io dtype, only with pre_weight) are dense;
 * either may be NULL (zero).  Writes dx, dgate (only with gate) io dtype,
 * d_residual (residual dtype, only with residual), all dense; d_post_weight,
 * d_scale, d_pre_weight [width] fp32, each only with its input.  The sums over
 * rows are fp32 in a fixed order: repeats are bit-identical.  Stream-ordered
 * workspace of up to 3 * width floats for each row in work on the device.
 */
KDA_API kda_status kda_block_norm_bwd(
    const kda_norm_shape* shape, const void* x, const float* post_weight,
    const void* gate, const void* residual, const float* scale,
    const float* pre_weight, const void* d_out, const void* d_normed, void* dx,
    void* dgate, void* d_residual, float* d_post_weight, float* d_scale,
    float* d_pre_weight, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LAYER_H_ */
