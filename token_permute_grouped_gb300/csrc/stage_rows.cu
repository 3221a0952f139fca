// All rows of ataOut in expert-major order, for the gated block: what
// permute.cu does, started while the kernel before it ends and letting the
// kernel behind it start at once, with the segment table made by a whole block.
//
// HBM-bound where there are many rows; with few, bound by its chain of dependent
// reads: counts, table, row, store.  Training calls against the other kernel
// (us): 65,308 rows of 2048 x 1408 1515 / 1506, 20,000 of 4096 x 64 107 / 100.5,
// 5013 of 1032 x 328 92 / 89, 1062 of 2568 x 456 49 / 46.
#include <algorithm>

#include "ffn.h"
#include "pdl.cuh"
#include "plan.cuh"

namespace a2av {

namespace {

constexpr int kStageThreads = 256;
constexpr int kStageWarps = kStageThreads / 32;
// Blocks an SM (a training call of 20,000 rows of 4096 x 64: 100.5 us with 8, 104
// with 4; loads that are evicted first from L2 instead of kept out of L1 112).
constexpr int kStageBlocks = 8;
constexpr int kPieceVecs = 4;  // 16-byte vectors a lane copies at a time
static_assert(kStageThreads >= kMaxSegments, "a thread holds a count");

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// The segment table, by a block: thread i holds count i in both orders.
// Returns whether the counts are consistent, to every thread.
__device__ __forceinline__ bool block_segments(const int32_t *recvCounts, int W, int e, int64_t A, SegmentTable &t,
                                               int64_t (&sums)[kStageWarps], int32_t (&dst_sums)[kStageWarps]) {
    const int i = threadIdx.x, lane = i % 32, warp = i / 32, E = W * e;
    const int32_t c = i < E ? recvCounts[i] : 0;  // of segment (w, j) = (i / e, i % e)
    if (i < E) t.tmp[i % e * W + i / e] = c;
    __syncthreads();
    const int32_t d = i < E ? t.tmp[i] : 0;
    int64_t src = c;
    int32_t dst = d;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t s = __shfl_up_sync(0xffffffffu, src, off);
        const int32_t v = __shfl_up_sync(0xffffffffu, dst, off);
        if (lane >= off) {
            src += s;
            dst += v;
        }
    }
    if (lane == 31) {
        sums[warp] = src;
        dst_sums[warp] = dst;
    }
    const bool bad = __syncthreads_or(c < 0);
    int64_t src0 = 0, total = 0;
    int32_t dst0 = 0;
#pragma unroll
    for (int k = 0; k < kStageWarps; ++k) {
        if (k < warp) {
            src0 += sums[k];
            dst0 += dst_sums[k];
        }
        total += sums[k];
    }
    if (i < E) {
        t.src[i] = static_cast<int32_t>(src0 + src - c);
        t.dst[i] = dst0 + dst - d;
    }
    if (i == 0) t.dst[E] = static_cast<int32_t>(total);
    __syncthreads();
    return !bad && total == A;
}

__global__ void __launch_bounds__(kStageThreads) stage_rows_kernel(const StageRowsLaunch p) {
    __shared__ SegmentTable table;
    __shared__ int64_t sums[kStageWarps];
    __shared__ int32_t dst_sums[kStageWarps];
    pdl_wait();
    // Cleared before the kernel behind this one can set bits of it.
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.status = 0;
        __threadfence();
    }
    if (blockIdx.x == 0) __syncthreads();
    pdl_trigger();
    const bool good = block_segments(p.recvCounts, p.W, p.e, p.A, table, sums, dst_sums);
    if (!good) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadCounts);
        return;
    }
    const int vpr = p.H1 / 8, ppr = (vpr + 32 * kPieceVecs - 1) / (32 * kPieceVecs);  // vectors and pieces of a row
    const int lane = threadIdx.x % 32, nwarps = gridDim.x * kStageWarps;
    const int64_t items = static_cast<int64_t>(p.A) * ppr;
    for (int64_t i = blockIdx.x * kStageWarps + threadIdx.x / 32; i < items; i += nwarps) {
        const int row = ppr == 1 ? static_cast<int>(i) : static_cast<int>(i / ppr);
        const int v0 = static_cast<int>(i - static_cast<int64_t>(row) * ppr) * 32 * kPieceVecs + lane;
        const int64_t from = source_row_in(table, p.W, p.e, segment_of(table, p.W, p.e, row), row);
        const uint4 *in = static_cast<const uint4 *>(p.src) + from * vpr;
        uint4 *out = static_cast<uint4 *>(p.dst) + static_cast<int64_t>(row) * vpr;
        uint4 r[kPieceVecs];
#pragma unroll
        for (int k = 0; k < kPieceVecs; ++k)
            if (v0 + 32 * k < vpr) r[k] = ld_stream(in + v0 + 32 * k);
#pragma unroll
        for (int k = 0; k < kPieceVecs; ++k)
            if (v0 + 32 * k < vpr) out[v0 + 32 * k] = r[k];
    }
}

}  // namespace

cudaError_t launch_stage_rows(const StageRowsLaunch &p, int sms, cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.A) * ((p.H1 / 8 + 32 * kPieceVecs - 1) / (32 * kPieceVecs));
    const int64_t blocks = std::min<int64_t>((items + kStageWarps - 1) / kStageWarps, static_cast<int64_t>(sms) * kStageBlocks);
    return launch_pdl(stage_rows_kernel, static_cast<unsigned>(std::max<int64_t>(blocks, 1)), kStageThreads, 0, 0, stream,
                      p);
}

}  // namespace a2av
