// Host-side launch descriptions of the grouped product of 8-bit rows with a
// float32 scale per 128 (a2av_gmm_g128.h; internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace a2av {

struct G128Launch {
    const int32_t *recvCounts;
    int32_t W, e, A, K, N;
    int32_t qtype;          // 0 E4M3FN, 1 E5M2
    const float *xs, *ws;   // scales of the arrival rows and of the weights
    void *y;
    int32_t *status;
    int32_t write_status;
    int32_t after_permute;  // launched to overlap the kernel before it, which stages the rows
    int32_t direct_halves;  // halves inside one segment are read in place from ataOut
    int32_t bn;             // columns of a tile: 256 or 128
    int32_t grid;           // CTAs, two a cluster
    uint64_t wait_limit_ns;
    CUtensorMap tmA;        // expert-major codes [A, K], box 128 x 128 rows
    CUtensorMap tmDirect;   // ataOut codes, likewise
    CUtensorMap tmB;        // weight codes [e, N, K], box 128 x bn / 2 columns
};
cudaError_t launch_g128_gemm(const G128Launch &p, bool bf16, cudaStream_t stream);
int g128_gemm_max_clusters();

}  // namespace a2av
