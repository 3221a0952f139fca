/*
 * a2av_ffn — the operators around the grouped product of an expert layer, on
 * one GB300: the RMS norm in front of the dispatch, the gated feed-forward
 * block of the experts, the gated activation between two block-scaled
 * products, and the gradients of the norm, the block and the grouped product.
 *
 * Conventions are those of a2av_gmm.h: plain device pointers, row-major
 * layouts, the caller owns every buffer, nothing is allocated, kept or
 * synchronised, work is only enqueued on `stream`, every call returns a
 * status code, and the same inputs give bitwise the same outputs (sums run in
 * a fixed order).  Outputs do not overlap inputs or each other, but where a
 * call says that they may.  Element type T: bf16 or fp16 (a2av_dtype), the
 * same for every T tensor of a call.  Sums, statistics and activations
 * are computed in fp32; each T output is rounded once (nearest even).
 *
 * Errors, for every call: A2AV_ERR_NULLPTR for a missing required pointer,
 * A2AV_ERR_INVALID for a shape, range, type or mode outside the limits given
 * here, A2AV_ERR_UNSUPPORTED for a width, stride or pointer this library
 * cannot take (alignment), A2AV_ERR_WORKSPACE for a workspace that is too
 * small or not 256-byte aligned, A2AV_ERR_CUDA when a launch fails.
 *
 * 8-bit outputs (codes and scales) are in the formats a2av_gmm_mx.h and
 * a2av_quant_reduce.h read.  For a row v of fp32 values:
 *   A2AV_QMODE_MX        E4M3FN or E5M2 codes, one E8M0 scale byte E + 127 for
 *                        32 consecutive values: E = floor(log2(amax)) - emax
 *                        clamped to [-127, 127] (emax 8 for E4M3FN, 15 for
 *                        E5M2; E = -127 for amax = 0), code = v * 2^-E
 *   A2AV_QMODE_GROUP128  E4M3FN, E5M2 or INT8 codes, one float32 scale
 *                        m / qmax for 128 consecutive values, m =
 *                        max(amax, 2^-100), qmax 448, 57344 or 127,
 *                        code = v * (qmax / m)
 * codes rounded to nearest even and saturating at the largest finite value.
 * A block that holds an infinity or a NaN gets a NaN scale (E8M0 0xFF) and NaN
 * codes (INT8: 0).
 */
#ifndef A2AV_FFN_H
#define A2AV_FFN_H

#include <stddef.h>
#include <stdint.h>

#include "a2av_gmm.h"
#include "a2av_quant_reduce.h"

#ifdef __cplusplus
extern "C" {
#endif

#define A2AV_Q_NONE (-1) /* qtype of a call without an 8-bit output */

typedef enum {
    A2AV_ACT_SILU = 0,     /* g / (1 + e^-g) */
    A2AV_ACT_GELU_TANH = 1 /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
} a2av_act;

/*
 * RMS norm with the residual's addition and an 8-bit output:
 *
 *     s = x + residual                      (s = x without a residual)
 *     rstd = 1 / sqrt(mean(s^2) + eps)      over the H values of a row
 *     y = s * rstd * gamma
 *
 * Outputs, each written when its pointer is not NULL (one at least): h = s
 * rounded to T (the residual stream the layer passes on), y rounded to T,
 * codes and scales of the unrounded y (both or neither, by qtype), rstd.
 *
 *   x [rows, H], residual [rows, H]  T; rows x_stride, residual_stride
 *                                    elements apart (>= H; a residual stride
 *                                    of 0 adds one row to every row)
 *   gamma [H] T; h, y [rows, H] T; codes [rows, H] bytes;
 *   scales [rows, H/32] E8M0 bytes (MX) or [rows, H/128] float32 (GROUP128);
 *   rstd [rows] float32
 * h may be x or residual itself when that tensor's rows are H apart.
 *
 * Limits: 0 <= rows <= 2^31 - 1, 0 < H < 65536, H and the strides multiples of
 * 8, H a multiple of 32 (MX) or 128 (GROUP128) with an 8-bit output; T
 * tensors 16-byte aligned, codes 8-byte, float32 4-byte aligned.
 */
typedef struct {
    int64_t rows, H;
    int64_t x_stride, residual_stride; /* elements from one row to the next */
    int32_t dtype;                     /* a2av_dtype: bf16 or fp16 */
    int32_t qtype;                     /* a2av_qtype, or A2AV_Q_NONE */
    int32_t qmode;                     /* a2av_qmode */
    float eps;                         /* >= 0 */
} a2av_rms_norm_desc;

a2av_status a2av_rms_norm(const a2av_rms_norm_desc *desc, const void *x, const void *residual,
                          const void *gamma, void *h, void *y, void *codes, void *scales, float *rstd,
                          a2av_stream_t stream);

/*
 * Gradient of y = h * rstd * gamma with respect to h and gamma (rstd a
 * function of h), plus the gradient dh that reaches h directly:
 *
 *     a = dy * gamma,  n = h * rstd
 *     dx = dh + rstd * (a - n * mean(a * n))    (dh = 0 when it is NULL)
 *     dgamma = sum over rows of dy * n
 *
 * dx is the gradient of x and of the residual alike.  Through the 8-bit output
 * the gradient passes as through y (straight-through).
 *   dy, dh, h, dx [rows, H] T, contiguous; gamma [H] T; rstd [rows] float32;
 *   dgamma [H] float32.  dx may be dh or dy itself.  dgamma NULL: not computed.
 * Phase 1 gives the workspace (per-block partial sums of dgamma; 0 bytes for a
 * few rows, workspace may then be NULL).
 * Limits as above (H a multiple of 8), but dgamma 16-byte aligned.
 */
a2av_status a2av_rms_norm_backward_workspace_size(int64_t rows, int64_t H, int32_t dtype, size_t *bytes);
a2av_status a2av_rms_norm_backward(int64_t rows, int64_t H, int32_t dtype, const void *dy, const void *dh,
                                   const void *h, const void *gamma, const float *rstd, void *dx,
                                   float *dgamma, void *workspace, size_t workspace_bytes,
                                   a2av_stream_t stream);

/*
 * Gated activation with an 8-bit output: v = act(gate) * up, written as T
 * (h, optional) and as codes and scales (both or neither, by qtype).  Between
 * two block-scaled products: the first one's gate and up columns in, the
 * second one's operand out.
 *   gate, up [rows, N] T, rows `stride` elements apart (>= N; the two halves of
 *   a [rows, 2N] product have stride 2N); h [rows, N] T; codes, scales as above.
 * Limits: 0 <= rows <= 2^31 - 1, 0 < N < 65536, N and stride multiples of 8, N
 * a multiple of 32 (MX) or 128 (GROUP128) with an 8-bit output; alignments as for
 * a2av_rms_norm.
 */
typedef struct {
    int64_t rows, N, stride;
    int32_t dtype, act, qtype, qmode;
} a2av_glu_desc;

a2av_status a2av_glu_quant(const a2av_glu_desc *desc, const void *gate, const void *up, void *h, void *codes,
                           void *scales, a2av_stream_t stream);

/*
 * Gated feed-forward block over ragged experts: both projections, the
 * activation and their product in one kernel,
 *
 *     G = permuteOut x gateWeight,  U = permuteOut x upWeight   (per expert)
 *     h = act(G) * U
 *
 * on the rows and counts a2av_gmm_run takes: ataOut [A, H1] rank-major,
 * recvCounts [W * e]; permuteOut [A, H1] expert-major is written when
 * want_permute_out is set (the backward pass needs it).  With W = 1 the rows
 * are expert-major as they arrive, ataOut is used as permuteOut, and
 * want_permute_out must be 0.
 *   gateWeight, upWeight [e, H1, N] T; h [A, N] T (expert-major);
 *   saved [2, A, N] float32: the unrounded G, then U, for the backward pass
 *   (written when `save` is set).  They are kept in 32 bits because their
 *   rounding to T would nearly double the gradients' error.
 *
 * Backward, for a gradient dh [A, N] of h:
 *     dG = dh * U * act'(G),  dU = dh * act(G)      rounded to T, the type the
 *                                                   tensor cores multiply (A <= 32:
 *                                                   to the sum of two Ts)
 *     dPermuteOut = dG x gateWeight^T + dU x upWeight^T
 *     dGate = permuteOut^T x dG,  dUp = permuteOut^T x dU   per expert
 * Up to 32 rows in all, whatever their experts, a gradient's error is that of its
 * own rounding; beyond, the slopes' rounding makes it 1.4 times as large, and in
 * fp16 a slope above 65504 becomes an infinity, one below 2^-14 loses bits and
 * one below 2^-25 becomes 0.
 * dAtaOut [A, H1] holds dPermuteOut's rows back in rank-major order; dGate,
 * dUp [e, H1, N] (zero for an expert without rows).  dAtaOut may be NULL, and
 * so may dGate and dUp together.  permuteOut is what the forward call wrote
 * (W = 1: ataOut).
 *
 * Two phases, as in a2av_gmm.h; one workspace serves both directions, and
 * a2av_gmm_read_device_status reads the device status of the last call on it.
 * Limits: those of a2av_gmm.h (W * e <= 256, e <= 32, H1, N < 65536 and
 * multiples of 8, A <= 2^31 - 1); T tensors 16-byte, saved 32-byte, recvCounts
 * 4-byte aligned.
 */
typedef struct {
    int32_t W, e;
    int64_t A, H1, N;
    int32_t dtype;            /* a2av_dtype: bf16 or fp16 */
    int32_t act;              /* a2av_act */
    int32_t want_permute_out; /* nonzero: permuteOut is written (W > 1 only) */
    int32_t save;             /* nonzero: saved is written, for the backward pass */
} a2av_gated_desc;

a2av_status a2av_gated_workspace_size(const a2av_gated_desc *desc, size_t *bytes);
a2av_status a2av_gated_run(const a2av_gated_desc *desc, const void *ataOut, const int32_t *recvCounts,
                           const void *gateWeight, const void *upWeight, void *permuteOut, void *h,
                           float *saved, void *workspace, size_t workspace_bytes, a2av_stream_t stream);
a2av_status a2av_gated_backward(const a2av_gated_desc *desc, const void *dh, const void *permuteOut,
                                const int32_t *recvCounts, const void *gateWeight, const void *upWeight,
                                const float *saved, void *dAtaOut, void *dGate, void *dUp, void *workspace,
                                size_t workspace_bytes, a2av_stream_t stream);

/*
 * Gradients of the grouped product gmmY = permuteOut x gmmWeight of a2av_gmm.h:
 *
 *     dPermuteOut = dY x gmmWeight^T            per expert
 *     dWeight = permuteOut^T x dY               per expert
 *
 * desc as for a2av_gmm_run, with BS = 0 (a shared expert's gradients are a
 * call of their own with W = e = 1); want_permute_out, path and tiles are not
 * looked at.  dY [A, N1] expert-major, permuteOut [A, H1]; dAtaOut [A, H1]:
 * dPermuteOut's rows back in rank-major order; dWeight [e, H1, N1].  Either
 * output may be NULL.  The workspace holds the device status word and, where a
 * gradient has few tiles over a long contraction, the float32 sums of the
 * contraction's slices, which are added in order.
 */
a2av_status a2av_gmm_backward_workspace_size(const a2av_gmm_desc *desc, size_t *bytes);
a2av_status a2av_gmm_backward(const a2av_gmm_desc *desc, const void *dY, const void *permuteOut,
                              const int32_t *recvCounts, const void *gmmWeight, void *dAtaOut, void *dWeight,
                              void *workspace, size_t workspace_bytes, a2av_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* A2AV_FFN_H */
