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
};
// kind: quant_kind() of the 8-bit output, or -1.
cudaError_t launch_rms_norm(const RmsNormLaunch &p, bool bf16, int kind, int sms, cudaStream_t stream);

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
    uint64_t inv64;  // set by the launch: 2^64 and 2^32 over N / 8, rounded up
    uint32_t inv32;
};
cudaError_t launch_glu_quant(GluLaunch p, bool bf16, int act, int kind, cudaStream_t stream);

// All rows in expert-major order; clears the status word (stage_rows.cu).
struct StageRowsLaunch {
    const int32_t *recvCounts;
    int32_t W, e, A, H1;
    const void *src;
    void *dst;
    int32_t *status;
};
cudaError_t launch_stage_rows(const StageRowsLaunch &p, int sms, cudaStream_t stream);

// dG = dh U act'(G), dU = dh act(G) for [rows, N] values.
struct GluGradLaunch {
    int32_t rows, N;
    const void *dh;
    const float *gate, *up;
    void *dgate, *dup;
    int64_t low;      // 16-byte vectors from a slope's first summand to its second (0: one summand, the rounded slope)
    int32_t *pieces;  // counts of finished pieces by 128 rows, zero at the start, for a GEMM that runs beside
                      // this kernel; NULL: not counted, and the kernel takes the SMs for itself
};
int glu_grad_pieces(int64_t rows, int64_t N);  // pieces of a block of this many (up to 128) rows
cudaError_t launch_glu_grad(const GluGradLaunch &p, bool bf16, int act, int sms, cudaStream_t stream);

// The products of a gated block (grad 0) or the gradients of one or two
// products over the same rows (grad 1), over ragged expert groups
// (expert_gemm.cu).
struct ExpertGemmLaunch {
    const int32_t *recvCounts;
    int32_t W, e, A;
    int32_t bf16, grad, act;
    // Tiles over the experts' rows: gated [A, N] = [A, K] x [K, N] twice;
    // gradient [A, N] = sum over phases of [A, K] x [N, K]^T.  N 0: none.
    int32_t K, N, phases;
    int32_t parts;          // gradients: 2 where each D_p comes as two summands
    int32_t one_a, one_b;   // 1: a stage's operand is one TMA load (4-D map), 0: two (3-D map)
    int32_t direct_halves;  // gated: halves inside one segment are read in place from ataOut
    // Tiles of the weights' gradients, [wM, wN] an expert = X^T D.  wM 0: none.
    int32_t wM, wN;
    int32_t one_x;
    int32_t half_step;      // columns from a tile's first accumulator half to its second: bn / 2 where both
                            // halves belong to one matrix, 0 where the second half is another matrix
    int32_t bn;             // accumulator columns of a tile: 256 or 128
    const int32_t *pieces;  // gradient: the D_p are in the making beside this kernel (glu_grad.cu)
    int32_t row_pieces, last_pieces;  // pieces of 128 rows; of the last block of A
    int32_t after_permute;  // gated: launched to overlap the kernel before it, which stages the rows
    int32_t *status;
    int32_t write_status;
    int32_t grid;           // CTAs, two a cluster
    uint64_t wait_limit_ns;
    void *out, *out_w[2];   // over the rows; weights' gradients by accumulator half
    // Gradients: equal slices that the contraction of a tile over rows, and of a weights' gradient, is cut into.
    // Above 1, a slice's sums go to part [slices][A][N] or part_w [matrix][w_slices][e][wM][wN] and a second kernel
    // adds them in order.
    int32_t slices, w_slices;
    float *part, *part_w;
    float *saved[2];        // gated: unrounded G and U, or NULL
    // tmA: the D_p by phase, then their second summands, as A; tmD: the same as B of the weights' gradient.
    CUtensorMap tmA[4], tmB[2], tmX, tmD[4];
    CUtensorMap tmDirect;
};
cudaError_t launch_expert_gemm(const ExpertGemmLaunch &p, cudaStream_t stream);
int expert_gemm_max_clusters();

// The gated block for a few rows (gated_rows.cu).
struct GatedRowsLaunch {
    const int32_t *recvCounts;
    int32_t W, e, A, K, N;
    void *h;
    float *saved[2];
    int32_t *status;
    uint64_t wait_limit_ns;
    int32_t after_permute;  // runs beside the kernel before it, which stages the rows and has cleared the status word
    int32_t split, grid;  // set by the launch: CTAs of a cluster, CTAs
    int32_t guess;        // likewise: experts taken to have rows before they are counted (all, or 0)
    const void *x;            // ataOut
    CUtensorMap tmGate, tmUp; // [e][K][N], box 64 columns x 128 k
};
// Rows the fullest of e experts is expected to have when A rows spread at random.
double gated_rows_most(int64_t A, int32_t e);
cudaError_t launch_gated_rows(GatedRowsLaunch p, bool bf16, int act, cudaStream_t stream);

}  // namespace a2av
