// Host-side launch descriptions of the expert layer for a few tokens
// (a2av_moe.h; internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "a2av_moe.h"

namespace a2av {

constexpr int kMoeTokens = 64;
constexpr int kMoeExperts = 256;
constexpr int kMoeChosen = 8;

// CTAs of the products: one an SM of a GB300.  Not asked of the device: the
// workspace's size depends on it, and is asked for without one.
constexpr int kMoeCtas = 152;

struct MoeRouterLaunch {
    int32_t T, E, H;
    const void *x, *router;  // [T, H], [E, H]
    float *logits;           // [T, E]
    int32_t *status;         // cleared
    int32_t *arrivals;       // [2][kMoeCtas], cleared
};
cudaError_t launch_moe_router(const MoeRouterLaunch &p, bool bf16, bool router32, cudaStream_t stream);

// What the choice of experts is made from.
struct MoeChoice {
    int32_t T, E, K, score, renormalise;
    float scale;
    const float *logits, *bias;
    int32_t *experts;  // [T, K], or NULL
    float *weights;    // likewise
    int2 *chosen;      // [T, K]: expert and weight, for the products
};
cudaError_t launch_moe_choose(const MoeChoice &c, cudaStream_t stream);

struct MoeRowsLaunch {
    MoeChoice choice;
    int32_t H, N;
    const void *residual;
    void *h;             // [2][T * K][N]: the gated block's values, expert after expert, in two summands (value_parts)
    void *y;
    int32_t *status;
    uint64_t wait_limit_ns;
    int32_t stages;      // set by the launch
    int32_t joined;      // likewise: the second product's shares are added by a kernel behind it
    int32_t *units;      // of the second product, for that kernel
    float *sums;         // [kMoeCtas][2][T][256 or 128]: shares of jobs that several CTAs have
    int32_t *arrivals;   // [kMoeCtas], 0: of those CTAs, by the first
    CUtensorMap tmA[2];  // gate and up [E][H][N], or down [E][N][H] (the first): box 64 columns x 64
    CUtensorMap tmX;     // x [1][T][H], or h [2][T * K][N]: box 64 x moe_unit_rows() x all
};
// Rows that a product takes at a time: 16, 32 or 64.
int moe_unit_rows(int T, int E, int K, bool down);
cudaError_t launch_moe_gated(MoeRowsLaunch p, bool bf16, int act, cudaStream_t stream);
cudaError_t launch_moe_down(MoeRowsLaunch p, bool bf16, cudaStream_t stream);

}  // namespace a2av
