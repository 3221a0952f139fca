// Host-side launch descriptions of the grouped product of 8-bit rows with a
// float32 scale per 128 (a2av_gmm_g128.h; internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace a2av {

// CTAs of the few-row kernel: one an SM of a GB300.  Not asked of the device: the
// workspace's size depends on it, and is asked for without one.
constexpr int kG128Ctas = 152;
constexpr int kG128UnitRows = 16;  // rows that it takes at a time

struct G128Launch {
    const int32_t *recvCounts;
    int32_t W, e, A, K, N;
    int32_t qtype;          // 0 E4M3FN, 1 E5M2
    const float *xs, *ws;   // scales of the arrival rows (few-row kernel: those of G128Stage) and of the weights
    void *y;
    int32_t *status;
    int32_t write_status;
    int32_t after_permute;  // launched to overlap the kernel before it, which stages the rows
    int32_t direct_halves;  // halves inside one segment are read in place from ataOut
    int32_t pair;           // tiles of 256 x 256 on two CTAs, or of 128 x 128 on one
    int32_t grid;           // CTAs
    uint64_t wait_limit_ns;
    // The few-row kernel's:
    float *sums;            // [kG128Ctas][2][kG128UnitRows][128]: shares of jobs that several CTAs have
    int32_t *arrivals;      // [kG128Ctas], 0: of those CTAs, by the first
    CUtensorMap tmA;        // expert-major codes [A, K], box 128 x 128 (few-row kernel: 16) rows
    CUtensorMap tmDirect;   // ataOut codes, likewise
    CUtensorMap tmB;        // weight codes [e, N, K], box 128 x 128 columns
};
cudaError_t launch_g128_gemm(const G128Launch &p, bool bf16, cudaStream_t stream);
int g128_gemm_max_clusters();

// For few rows an expert (g128_rows.cu), behind the kernel that stages them.
struct G128Stage {
    const int32_t *recvCounts;
    int32_t W, e, A, K;
    const void *src;    // arrival rows' codes
    const float *xs;    // and scales
    void *dst;          // codes in expert-major order, or NULL: not wanted
    float *scales;      // [K / 128][A], rows in expert-major order
    int32_t *status;    // cleared
    int32_t *arrivals;  // likewise
};
cudaError_t launch_g128_stage(const G128Stage &p, cudaStream_t stream);
cudaError_t launch_g128_rows(const G128Launch &p, bool bf16, cudaStream_t stream);

}  // namespace a2av
