// The router's logits of the expert layer for a few tokens: l[t][e] = sum over h
// of x[t][h] router[e][h].
//
// A block holds a few experts' and tokens' rows against each other, its threads
// taking vectors of 8 along H in turn; their fp32 sums are joined with the
// rounding errors carried along, since a logit's last digits may decide a choice.
// Bound by latency for one token (a block an expert; the rows' way from HBM), by
// the reads of the rows from L2 for many.
#include "activation.cuh"
#include "moe.h"
#include "pdl.cuh"
#include "rows.cuh"

namespace a2av {

namespace {

constexpr int kRouterThreads = 256;
constexpr int kRouterWarps = kRouterThreads / 32;

__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// R32: the router is float32.  NE, NT: experts and tokens of a block.
template <bool BF16, bool R32, int NE, int NT>
__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeRouterLaunch p) {
    __shared__ float2 sums[kRouterWarps][NE * NT];
    const int e0 = blockIdx.x * NE, t0 = blockIdx.y * NT, vecs = p.H / 8;
    constexpr int kVec = R32 ? 32 : 16;  // bytes of 8 router values
    const auto router_at = [&](int e, int v) {
        return static_cast<const uint8_t *>(p.router) + (static_cast<size_t>(e) * vecs + v) * kVec;
    };
    // The weights' way to L2 begins while the kernel before this one ends.
    for (int i = 0; i < NE && e0 + i < p.E; ++i)
        for (int v = threadIdx.x * (128 / kVec); v < vecs; v += kRouterThreads * (128 / kVec)) prefetch_l2(router_at(e0 + i, v));
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0;
    f32x2 acc[NE][NT];
#pragma unroll
    for (int i = 0; i < NE; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = 0;
    for (int v = threadIdx.x; v < vecs; v += kRouterThreads) {
        f32x2 x[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint4 raw = t0 + j < p.T
                                  ? *(static_cast<const uint4 *>(p.x) + static_cast<size_t>(t0 + j) * vecs + v)
                                  : make_uint4(0, 0, 0, 0);
            unpack8<BF16>(raw, x[j]);
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            f32x2 w[4] = {0, 0, 0, 0};
            if (e0 + i < p.E) {
                if constexpr (R32) {
                    const float4 *r = reinterpret_cast<const float4 *>(router_at(e0 + i, v));
                    const float4 a = r[0], b = r[1];
                    w[0] = pair_of(a.x, a.y), w[1] = pair_of(a.z, a.w), w[2] = pair_of(b.x, b.y), w[3] = pair_of(b.z, b.w);
                } else {
                    unpack8<BF16>(*reinterpret_cast<const uint4 *>(router_at(e0 + i, v)), w);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][j] = fma2(x[j][k], w[k], acc[i][j]);
        }
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float a, b;
            split(acc[i][j], a, b);
            float hi = a, lo = 0.0f;
            two_sum(hi, lo, b, 0.0f);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                two_sum(hi, lo, __shfl_xor_sync(0xffffffffu, hi, off), __shfl_xor_sync(0xffffffffu, lo, off));
            if (lane == 0) sums[warp][i * NT + j] = make_float2(hi, lo);
        }
    }
    __syncthreads();
    if (threadIdx.x < NE * NT) {
        const int i = threadIdx.x / NT, j = threadIdx.x % NT;
        float hi = 0.0f, lo = 0.0f;
        for (int w = 0; w < kRouterWarps; ++w) two_sum(hi, lo, sums[w][threadIdx.x].x, sums[w][threadIdx.x].y);
        if (e0 + i < p.E && t0 + j < p.T)
            p.logits[(t0 + j) * p.E + e0 + i] = fabsf(hi) < __uint_as_float(0x7f800000u) ? hi + lo : hi;
    }
}

template <bool BF16, bool R32>
cudaError_t launch_type(const MoeRouterLaunch &p, cudaStream_t stream) {
    if (p.T == 0)  // nothing but the status
        return launch_pdl(moe_router_kernel<BF16, R32, 1, 1>, dim3(1, 1), kRouterThreads, 0, 0, stream, p);
    if (p.T == 1)
        return launch_pdl(moe_router_kernel<BF16, R32, 1, 1>, dim3(p.E, 1), kRouterThreads, 0, 0, stream, p);
    return launch_pdl(moe_router_kernel<BF16, R32, 4, 4>, dim3((p.E + 3) / 4, (p.T + 3) / 4), kRouterThreads, 0, 0, stream,
                      p);
}

}  // namespace

cudaError_t launch_moe_router(const MoeRouterLaunch &p, bool bf16, bool router32, cudaStream_t stream) {
    if (router32) return bf16 ? launch_type<true, true>(p, stream) : launch_type<false, true>(p, stream);
    return bf16 ? launch_type<true, false>(p, stream) : launch_type<false, false>(p, stream);
}

}  // namespace a2av
