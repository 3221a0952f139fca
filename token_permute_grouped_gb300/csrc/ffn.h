// Host-side launch descriptions of the expert-layer operators declared in
// a2av_ffn.h (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "a2av_ffn.h"

namespace a2av {

struct RmsNormLaunch {
    int32_t rows, H;
    int64_t x_stride, r_stride;  // elements
    const void *x, *residual, *gamma;
    void *h, *y;
    uint8_t *codes;
    void *scales;
    float *rstd;
    float eps;
    int32_t qtype;
};
cudaError_t launch_rms_norm(const RmsNormLaunch &p, bool bf16, int qmode, int sms, cudaStream_t stream);

struct RmsNormGradLaunch {
    int32_t rows, H;
    const void *dy, *dh, *h, *gamma;
    const float *rstd;
    void *dx;
    float *dgamma;
    float *partial;  // [blocks, H]
    int32_t blocks;
};
// Blocks the gradient kernel runs for this shape, each with a row of partial sums of dgamma.
int rms_norm_grad_blocks(int64_t rows, int64_t H);
cudaError_t launch_rms_norm_grad(const RmsNormGradLaunch &p, bool bf16, cudaStream_t stream);

struct GluLaunch {
    int64_t rows;
    int32_t N;
    int64_t stride;
    const void *gate, *up;
    void *h;
    uint8_t *codes;
    void *scales;
    int32_t qtype;
};
cudaError_t launch_glu_quant(const GluLaunch &p, bool bf16, int act, int qmode, int sms, cudaStream_t stream);

// dG = dh U act'(G), dU = dh act(G), element by element over n values.
struct GluGradLaunch {
    int64_t n;  // multiple of 8
    const void *dh;
    const float *gate, *up;
    void *dgate, *dup;
};
cudaError_t launch_glu_grad(const GluGradLaunch &p, bool bf16, int act, int sms, cudaStream_t stream);

// The three products of a gated block or of a grouped product's gradient, as
// one kernel over ragged expert groups (expert_gemm.cu).
enum ExpertForm {
    kFormGated = 0,      // h = act(X Wg) * (X Wu)
    kFormGradRows = 1,   // dX = sum over p of D_p W_p^T
    kFormGradWeight = 2  // dW = X^T D, contracted over an expert's rows
};

struct ExpertGemmLaunch {
    const int32_t *recvCounts;
    int32_t W, e, A;
    int32_t K;           // contraction length (rows' gradient: of one phase; weights' gradient: unused)
    int32_t phases;      // rows' gradient: products added into one accumulator (gated 2, plain 1)
    int32_t M, N;        // weights' gradient: rows of dW; N: output columns
    int32_t half_step;   // columns from a tile's first accumulator half to its second: 128 where both
                         // halves belong to one matrix, 0 where the second half is another matrix
    int32_t one_a, one_b;  // 1: a stage's operand is one TMA load (4-D map), 0: two (3-D map)
    int32_t bf16, form, act;
    int32_t *status;
    int32_t write_status;
    int32_t direct_halves;  // gated: halves inside one segment are read in place from ataOut
    int32_t after;          // launched beside the kernel before it (programmatic dependent launch)
    int32_t grid;           // CTAs, two a cluster
    uint64_t wait_limit_ns;
    void *out[2];           // by accumulator half
    float *saved[2];        // gated: unrounded G and U, or NULL
    CUtensorMap tmA[2], tmB[2], tmY[2];
    CUtensorMap tmDirect;
};
cudaError_t launch_expert_gemm(const ExpertGemmLaunch &p, cudaStream_t stream);
int expert_gemm_max_clusters();

}  // namespace a2av
