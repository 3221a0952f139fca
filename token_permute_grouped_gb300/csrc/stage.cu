// The kernels that make the rows a GEMM of expert_gemm.cu reads: the
// expert-major copy of rank-major rows, and the gated block's element-wise
// gradient dG = dh U act'(G), dU = dh act(G).
//
// Both are HBM-bound while the GEMM behind them is tensor-bound, so the two run
// side by side: these take at most two blocks of 256 threads an SM, which fit
// beside a GEMM CTA (219 KB of shared memory, 44 K registers), work through the
// rows in the order the GEMM does, and count the finished pieces of each 128
// rows, for which the GEMM's producer waits.  They never wait for the GEMM,
// and all their blocks are resident before it starts, so it cannot hold them up.
#include <algorithm>

#include "activation.cuh"
#include "ffn.h"
#include "pdl.cuh"
#include "plan.cuh"

namespace a2av {

namespace {

constexpr int kStageThreads = 256;
constexpr int kStageWarps = kStageThreads / 32;
#ifndef ROWS_PER_SM
#define ROWS_PER_SM 64
#define GRAD_PER_SM 8
#endif
constexpr int kRows = 128;         // rows of a counted block
constexpr int kChunkVecs = 128;    // 16-byte vectors of a row in a piece of the copy: 2 KB
constexpr int kFlatVecs = 2048;    // vectors of a piece of the gradient

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// The block's stores of this piece are done: one more finished piece of `count`.
__device__ __forceinline__ void count_piece(int32_t *count) {
    __syncthreads();
    if (threadIdx.x == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(count) : "memory");
}

__global__ void __launch_bounds__(kStageThreads) stage_rows_kernel(const StageRowsLaunch p) {
    __shared__ SegmentTable seg;
    __shared__ int32_t half0[kMaxExperts + 1];
    __shared__ int ok;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_wait();
    if (blockIdx.x == 0) {  // before any later kernel sets a bit in it
        if (threadIdx.x == 0) {
            *p.status = 0;
            __threadfence();
        }
        __syncthreads();
    }
    pdl_trigger();
    if (warp == 0) {
        const bool good = build_segment_table(p.recvCounts, p.W, p.e, p.A, seg, lane);
        int halves = 0;
        if (lane < p.e && good) halves = (seg.dst[(lane + 1) * p.W] - seg.dst[lane * p.W] + kRows - 1) / kRows;
        int inc = halves;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane < p.e) half0[lane] = inc - halves;
        if (lane == 31) half0[p.e] = inc;
        if (lane == 0) {
            ok = good;
            if (blockIdx.x == 0 && !good) atomicOr(p.status, kStatusBadCounts);
        }
    }
    __syncthreads();
    if (!ok) return;
    const int vpr = p.H1 / 8, chunks = (vpr + kChunkVecs - 1) / kChunkVecs;
    const int64_t items = static_cast<int64_t>(half0[p.e]) * chunks;
    int j = 0;  // the expert of the half: halves come in ascending order
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int half = static_cast<int>(i / chunks), chunk = static_cast<int>(i - static_cast<int64_t>(half) * chunks);
        while (half >= half0[j + 1]) ++j;
        const int g1 = seg.dst[(j + 1) * p.W];
        const int first = seg.dst[j * p.W] + (half - half0[j]) * kRows, end = min(first + kRows, g1);
        const bool straddles = !half_in_one_segment(seg, p.W, p.e, first, g1);
        if (p.only_straddling && !straddles) continue;  // (the same for the whole block)
        const int v0 = chunk * kChunkVecs + lane;
        // Two rows a warp at a time: eight loads in flight a thread.
        for (int d = first + 2 * warp; d < end; d += 2 * kStageWarps) {
            uint4 r[2][kChunkVecs / 32];
            const uint4 *in[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                in[k] = static_cast<const uint4 *>(p.src) +
                        static_cast<size_t>(source_row(seg, p.W, p.e, min(d + k, end - 1))) * vpr;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int v = 0; v < kChunkVecs / 32; ++v)
                    if (d + k < end && v0 + 32 * v < vpr) r[k][v] = ld_stream(in[k] + v0 + 32 * v);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int v = 0; v < kChunkVecs / 32; ++v)
                    if (d + k < end && v0 + 32 * v < vpr)
                        static_cast<uint4 *>(p.dst)[static_cast<size_t>(d + k) * vpr + v0 + 32 * v] = r[k][v];
        }
        if (p.pieces && straddles) count_piece(p.pieces + half);
    }
}

// A block of 128 rows is contiguous in every tensor: its vectors are taken in
// pieces of kFlatVecs.
template <bool BF16, int ACT>
__global__ void __launch_bounds__(kStageThreads) glu_grad_kernel(const GluGradLaunch p) {
    pdl_wait();
    pdl_trigger();
    const int64_t per_block = static_cast<int64_t>(kRows) * (p.N / 8), total = static_cast<int64_t>(p.rows) * (p.N / 8);
    const int pieces = static_cast<int>((per_block + kFlatVecs - 1) / kFlatVecs);
    const int blocks = (p.rows + kRows - 1) / kRows;
    for (int64_t i = blockIdx.x; i < static_cast<int64_t>(blocks) * pieces; i += gridDim.x) {
        const int64_t block = i / pieces;
        const int64_t v0 = block * per_block + (i - block * pieces) * kFlatVecs;
        const int64_t end = min(min(v0 + kFlatVecs, (block + 1) * per_block), total);
        if (v0 >= end) continue;  // (the last block may have fewer pieces)
#pragma unroll 2
        for (int64_t v = v0 + threadIdx.x; v < end; v += kStageThreads) {
            const uint4 d = ld_stream(static_cast<const uint4 *>(p.dh) + v);
            const uint4 g0 = ld_stream(reinterpret_cast<const uint4 *>(p.gate) + 2 * v);
            const uint4 g1 = ld_stream(reinterpret_cast<const uint4 *>(p.gate) + 2 * v + 1);
            const uint4 u0 = ld_stream(reinterpret_cast<const uint4 *>(p.up) + 2 * v);
            const uint4 u1 = ld_stream(reinterpret_cast<const uint4 *>(p.up) + 2 * v + 1);
            const auto f = [](uint32_t a, uint32_t b) { return pair_of(__uint_as_float(a), __uint_as_float(b)); };
            const f32x2 g[4] = {f(g0.x, g0.y), f(g0.z, g0.w), f(g1.x, g1.y), f(g1.z, g1.w)};
            const f32x2 u[4] = {f(u0.x, u0.y), f(u0.z, u0.w), f(u1.x, u1.y), f(u1.z, u1.w)};
            f32x2 fd[4], dg[4], du[4];
            unpack8<BF16>(d, fd);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f32x2 slope;
                const f32x2 a = act_value_slope<ACT>(g[k], slope);
                dg[k] = mul2(mul2(fd[k], u[k]), slope);
                du[k] = mul2(fd[k], a);
            }
            static_cast<uint4 *>(p.dgate)[v] = pack8<BF16>(dg);
            static_cast<uint4 *>(p.dup)[v] = pack8<BF16>(du);
        }
        if (p.pieces) count_piece(p.pieces + block);
    }
}

// An SM's split of L1 and shared memory holds while blocks run on it, and a GEMM
// CTA needs the largest share, so a kernel that is to share its SMs asks for
// that share too (its own 3 KB would leave the SM set for L1, and the GEMM
// would start only as these blocks end).
template <typename Kernel>
cudaError_t beside_gemm(Kernel kern) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

}  // namespace

int stage_rows_pieces(int64_t H1) { return static_cast<int>((H1 / 8 + kChunkVecs - 1) / kChunkVecs); }

cudaError_t launch_stage_rows(const StageRowsLaunch &p, int sms, cudaStream_t stream) {
    const int64_t items = (static_cast<int64_t>(p.A) / kRows + p.e) * stage_rows_pieces(p.H1);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, static_cast<int64_t>(sms) * ROWS_PER_SM / 8));
    const cudaError_t err = beside_gemm(stage_rows_kernel);
    if (err != cudaSuccess) return err;
    return launch_pdl(stage_rows_kernel, grid, kStageThreads, 0, 0, stream, p);
}

int glu_grad_pieces(int64_t rows, int64_t N) {
    return static_cast<int>((rows * (N / 8) + kFlatVecs - 1) / kFlatVecs);
}

cudaError_t launch_glu_grad(const GluGradLaunch &p, bool bf16, int act, int sms, cudaStream_t stream) {
    const int64_t items = (static_cast<int64_t>(p.rows) + kRows - 1) / kRows * glu_grad_pieces(kRows, p.N);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, static_cast<int64_t>(sms) * GRAD_PER_SM / 8));
    const auto kern = bf16 ? (act == A2AV_ACT_SILU ? glu_grad_kernel<true, A2AV_ACT_SILU>
                                                   : glu_grad_kernel<true, A2AV_ACT_GELU_TANH>)
                           : (act == A2AV_ACT_SILU ? glu_grad_kernel<false, A2AV_ACT_SILU>
                                                   : glu_grad_kernel<false, A2AV_ACT_GELU_TANH>);
    const cudaError_t err = beside_gemm(kern);
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, grid, kStageThreads, 0, 0, stream, p);
}

}  // namespace a2av
