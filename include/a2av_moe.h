/*
 * a2av_moe — a whole expert layer for a few tokens (a decode step) on one GB300:
 * the router's choice, the chosen experts' gated blocks and down projections,
 * and their weighted sum,
 *
 *     l = x router^T                                 per token, E logits
 *     p = softmax(l) or 1 / (1 + e^-l)
 *     experts = the K largest of p + bias            (ties: the lowest index)
 *     w = p of the chosen, over their sum where `renormalise` is set, times scale
 *         (a ratio of scores, however small they are)
 *     y = residual + sum over k of w_k (act(x Wg_k) * (x Wu_k)) Wd_k
 *
 * Each expert's weights are read once for the tokens that chose it.  Larger
 * batches go through a2av_gated_run and a2av_gmm_run.  A call has four or five
 * kernels whose start and end take 20 to 30 us however small the experts are: for
 * less than about 30 MB of weights and more than a few tokens those two products,
 * with a router of the caller's own, may be the better path (64 tokens, 4 of 4
 * experts of 3288 x 192: 70 us, the two products 30).
 *
 *   x, residual, y [T, H] T (residual may be NULL: 0; y may be x or residual)
 *   router [E, H] T or float32; bias [E] float32 (may be NULL; it takes part in
 *   the choice only); gate, up [E, H, N] T; down [E, N, H] T
 *   experts [T, K] int32 and weights [T, K] float32, the largest p + bias first
 *   (either may be NULL)
 *
 * Element type T: bf16 or fp16.  Logits, scores, weights and sums are fp32; the
 * block's values go to the second product as two summands of T, which hold a value
 * to 2^-15 of it (bf16) or to 2^-22 of it or 2^-35, whichever is larger (fp16;
 * values beyond twice fp16's range are infinite).  So y's error is that of its own
 * rounding, in fp16 unless down or scale are large enough to bring values about
 * 2^-35 into it.  Without a bias the choice is made on the logits themselves.  A
 * NaN logit is chosen last; a token's NaN or infinity reaches no other token.
 *
 * Limits: 0 <= T <= 64, 1 <= E <= 256, 1 <= K <= 8, K <= E, 0 < H, N < 65536 and
 * multiples of 8; T tensors, router and bias 16-byte, experts and weights 4-byte
 * aligned.
 *
 * Two phases and conventions as in a2av_gmm.h; a2av_gmm_read_device_status reads
 * the device status of the last call on a workspace, which serves one call at a
 * time.
 */
#ifndef A2AV_MOE_H
#define A2AV_MOE_H

#include <stddef.h>
#include <stdint.h>

#include "a2av_ffn.h"
#include "a2av_gmm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { A2AV_SCORE_SOFTMAX = 0, A2AV_SCORE_SIGMOID = 1 } a2av_score;

typedef struct {
    int32_t T, E, K;
    int64_t H, N;
    int32_t dtype;        /* a2av_dtype: bf16 or fp16 */
    int32_t router_dtype; /* a2av_dtype: dtype, or A2AV_FP32 */
    int32_t act;          /* a2av_act */
    int32_t score;        /* a2av_score */
    int32_t renormalise;  /* nonzero: the chosen scores are divided by their sum */
    float scale;          /* finite */
} a2av_moe_desc;

a2av_status a2av_moe_workspace_size(const a2av_moe_desc *desc, size_t *bytes);
a2av_status a2av_moe_run(const a2av_moe_desc *desc, const void *x, const void *router, const float *bias,
                         const void *gate, const void *up, const void *down, const void *residual, void *y,
                         int32_t *experts, float *weights, void *workspace, size_t workspace_bytes,
                         a2av_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* A2AV_MOE_H */
