// The gated block's element-wise gradient, dG = dh U act'(G), dU = dh act(G):
// the operands of the GEMM behind it (expert_gemm.cu).
//
// HBM-bound while that GEMM is tensor-bound, so the two run side by side: one
// block of 256 threads an SM, which fits beside a GEMM CTA, works through the
// rows in the order the GEMM does and counts the finished pieces of each 128
// rows, for which the GEMM's producer waits.  This kernel never waits for the
// GEMM, and all its blocks are resident before the GEMM starts, so neither can
// hold up the other.  65,308 x 1408 values: 315 us alone with one block an SM
// (190 with eight, at the copy rate) and 905 us of GEMM; forward and backward of
// the gated block together take 1550 us side by side, 1715 one after the other
// (single calls after a pause; 1717 side by side in a loop, at the power limit).
#include <algorithm>

#include "activation.cuh"
#include "two_parts.cuh"
#include "ffn.h"
#include "pdl.cuh"

namespace a2av {

namespace {

constexpr int kGradThreads = 256;
constexpr int kRows = 128;         // rows of a counted block
constexpr int kFlatVecs = 2048;    // vectors of a piece

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

template <bool BF16>
__device__ __forceinline__ void two_parts8(const f32x2 (&v)[4], uint4 &high, uint4 &low) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a, b;
        uint32_t ha, la, hb, lb;
        split(v[k], a, b);
        two_parts<BF16>(a, ha, la);
        two_parts<BF16>(b, hb, lb);
        h[k] = ha | hb << 16;
        l[k] = la | lb << 16;
    }
    high = make_uint4(h[0], h[1], h[2], h[3]);
    low = make_uint4(l[0], l[1], l[2], l[3]);
}

// Counted, a block of 128 rows, which is contiguous in every tensor, is taken in
// pieces of kFlatVecs; otherwise all rows are one block and a piece is a vector
// a thread, so that few rows spread over the SMs (5013 x 328 values 9.5 us with
// pieces of kFlatVecs, 6 so).
template <bool BF16, int ACT>
__global__ void __launch_bounds__(kGradThreads) glu_grad_kernel(const GluGradLaunch p) {
    pdl_wait();
    pdl_trigger();
    const int64_t total = static_cast<int64_t>(p.rows) * (p.N / 8);
    const int64_t per_block = p.pieces ? static_cast<int64_t>(kRows) * (p.N / 8) : total;
    const int size = p.pieces ? kFlatVecs : kGradThreads;
    const int64_t pieces = (per_block + size - 1) / size, blocks = (total + per_block - 1) / per_block;
    for (int64_t i = blockIdx.x; i < blocks * pieces; i += gridDim.x) {
        const int64_t block = p.pieces ? i / pieces : 0;
        const int64_t v0 = block * per_block + (i - block * pieces) * size;
        const int64_t end = min(min(v0 + size, (block + 1) * per_block), total);
        if (v0 >= end) continue;  // (the last block may have fewer pieces)
#pragma unroll 2
        for (int64_t v = v0 + threadIdx.x; v < end; v += kGradThreads) {
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
            uint4 hg, hu;
            if (p.low) {
                uint4 lg, lu;
                two_parts8<BF16>(dg, hg, lg);
                two_parts8<BF16>(du, hu, lu);
                static_cast<uint4 *>(p.dgate)[p.low + v] = lg;
                static_cast<uint4 *>(p.dup)[p.low + v] = lu;
            } else {
                hg = pack8<BF16>(dg);
                hu = pack8<BF16>(du);
            }
            static_cast<uint4 *>(p.dgate)[v] = hg;
            static_cast<uint4 *>(p.dup)[v] = hu;
        }
        if (p.pieces) count_piece(p.pieces + block);
    }
}

// An SM's split of L1 and shared memory holds while blocks run on it, and a GEMM
// CTA needs the largest share, so a launch that is to share its SMs asks for that
// share too (otherwise the SM is set for L1, and the GEMM starts only as these
// blocks end).
constexpr int kBesideGemm = cudaSharedmemCarveoutMaxShared;

}  // namespace

int glu_grad_pieces(int64_t rows, int64_t N) {
    return static_cast<int>((rows * (N / 8) + kFlatVecs - 1) / kFlatVecs);
}

cudaError_t launch_glu_grad(const GluGradLaunch &p, bool bf16, int act, int sms, cudaStream_t stream) {
    const int64_t values = static_cast<int64_t>(p.rows) * p.N, per = 8 * kGradThreads;
    const int64_t items = p.pieces ? (static_cast<int64_t>(p.rows) + kRows - 1) / kRows * glu_grad_pieces(kRows, p.N)
                                   : (values + per - 1) / per;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, p.pieces ? sms : sms * 8));
    const auto kern = bf16 ? (act == A2AV_ACT_SILU ? glu_grad_kernel<true, A2AV_ACT_SILU>
                                                   : glu_grad_kernel<true, A2AV_ACT_GELU_TANH>)
                           : (act == A2AV_ACT_SILU ? glu_grad_kernel<false, A2AV_ACT_SILU>
                                                   : glu_grad_kernel<false, A2AV_ACT_GELU_TANH>);
    return launch_pdl(kern, grid, kGradThreads, 0, PdlShape(0, p.pieces ? kBesideGemm : -1), stream, p);
}

}  // namespace a2av
