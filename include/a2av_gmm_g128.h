/*
 * a2av_gmm_g128 — Permute + GroupedMatMul of 8-bit rows with a float32 scale
 * for each 128 values, on one GB300: the product that reads what a2av_rms_norm,
 * a2av_layer_norm and a2av_glu_quant write in A2AV_QMODE_GROUP128.
 *
 *     gmmY[i][n] = sum over blocks b of 128 of
 *         ataOut_s[i][b] * gmmWeight_s[j][n / 128][b] * sum over k in b of value(a[i][k]) * value(w[j][n][k])
 *
 * for the rows i of permuteOut = Permute(ataOut) that belong to expert j.  The
 * inner sums are the tensor cores' (tcgen05.mma kind::f8f6f4), accumulated in
 * fp32; each block's sum is scaled and added in fp32, the result rounded once to
 * the output type (nearest even).  A row's and a weight block's scale are
 * multiplied first: their product has to lie within fp32's range.
 *
 * Shapes and limits (as in a2av_gmm.h): W ranks, e local experts (1 <= e <= 32,
 * W * e <= 256), A rows (sum of recvCounts, 0 allowed, <= 2^31 - 1), 0 < H1, N1
 * < 65536; H1 a multiple of 128, N1 of 8.  A shared expert is a call of its own
 * with W = e = 1.
 *
 * Layouts (row-major, contiguous, device memory, 16-byte aligned; the float32
 * scales 4-byte aligned):
 *   ataOut_q    [A, H1]       codes, rank-major (as ataOut in a2av_gmm.h)
 *   ataOut_s    [A, H1/128]   float32 scales of those rows, same order
 *   recvCounts  [W * e]       int32
 *   gmmWeight_q [e, N1, H1]   codes: each output column's H1 codes contiguous
 *   gmmWeight_s [e, ceil(N1/128), H1/128]   float32, one for 128 columns x 128
 *                             codes (the last block of columns may be short)
 *   gmmY        [A, N1]       bf16 or fp16, expert-major
 *
 * Two phases and conventions as in a2av_gmm.h; a2av_gmm_read_device_status reads
 * the device status of the last call on a workspace.  The workspace serves one
 * call at a time.  Status codes: A2AV_ERR_NULLPTR, A2AV_ERR_INVALID (a shape,
 * type or format outside the limits), A2AV_ERR_UNSUPPORTED (widths or pointers
 * that this library cannot take), A2AV_ERR_WORKSPACE, A2AV_ERR_CUDA.
 */
#ifndef A2AV_GMM_G128_H
#define A2AV_GMM_G128_H

#include <stddef.h>
#include <stdint.h>

#include "a2av_gmm.h"
#include "a2av_quant_reduce.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t W, e;
    int64_t A, H1, N1;
    int32_t dtype; /* a2av_dtype of gmmY: bf16 or fp16 */
    int32_t qtype; /* a2av_qtype of rows and weights: E4M3FN or E5M2 */
} a2av_gmm_g128_desc;

a2av_status a2av_gmm_g128_workspace_size(const a2av_gmm_g128_desc *desc, size_t *bytes);
a2av_status a2av_gmm_g128_run(const a2av_gmm_g128_desc *desc, const void *ataOut_q, const float *ataOut_s,
                              const int32_t *recvCounts, const void *gmmWeight_q, const float *gmmWeight_s, void *gmmY,
                              void *workspace, size_t workspace_bytes, a2av_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* A2AV_GMM_G128_H */
