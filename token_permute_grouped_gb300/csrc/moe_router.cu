// The router's logits of the expert layer for a few tokens: l[t][e] = sum over h
// of x[t][h] router[e][h].
//
// A warp holds four experts' and four tokens' rows (one and one for a single
// token) against each other, or a part of them: `split` warps of a block take
// vectors of 8 along H in turn.  Their fp32 sums are joined with the rounding
// errors carried along, since a logit's last digits may decide a choice.  Bound by
// latency for few tokens, by the reads of the rows from L2 for many.
#include "activation.cuh"
#include "moe.h"
#include "moe_plan.cuh"
#include "pdl.cuh"
#include "rows.cuh"

namespace a2av {

namespace {

constexpr int kRouterThreads = 256;
constexpr int kRouterWarps = kRouterThreads / 32;

__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// Sums over a warp of the N values of each lane, N a power of two: a lane ends
// with that of value lane / (32 / N).  Each step hands half of what is left to
// the lane across.
template <int N>
__device__ __forceinline__ void warp_sums(float (&hi)[N], float (&lo)[N], int lane) {
    int off = 16;
#pragma unroll
    for (int n = N / 2; n > 0; n /= 2, off /= 2) {
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float h = upper ? hi[i] : hi[i + n], l = upper ? lo[i] : lo[i + n];
            if (upper) hi[i] = hi[i + n], lo[i] = lo[i + n];
            two_sum(hi[i], lo[i], __shfl_xor_sync(0xffffffffu, h, off), __shfl_xor_sync(0xffffffffu, l, off));
        }
    }
#pragma unroll
    for (; off > 0; off /= 2)
        two_sum(hi[0], lo[0], __shfl_xor_sync(0xffffffffu, hi[0], off), __shfl_xor_sync(0xffffffffu, lo[0], off));
}

// R32: the router is float32.  NE, NT: experts and tokens of a warp.
template <bool BF16, bool R32, int NE, int NT>
__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeRouterLaunch p, int split) {
    __shared__ float2 sums[kRouterWarps][NE * NT];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int tile = blockIdx.x * (kRouterWarps / split) + warp / split, sub = warp % split;
    const int etiles = (p.E + NE - 1) / NE;
    const int e0 = tile % etiles * NE, t0 = tile / etiles * NT, vecs = p.H / 8;
    constexpr int kVec = R32 ? 32 : 16;  // bytes of 8 router values
    const auto router_at = [&](int e, int v) {
        return static_cast<const uint8_t *>(p.router) + (static_cast<size_t>(e) * vecs + v) * kVec;
    };
    // The weights' way to L2 begins while the kernel before this one ends.
    if (t0 == 0) {
        constexpr int kLine = 128 / kVec;
        for (int i = 0; i < NE && e0 + i < p.E; ++i)
            for (int v = (sub * 32 + lane) * kLine; v < vecs; v += split * 32 * kLine) prefetch_l2(router_at(e0 + i, v));
    }
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *p.status = 0;
        for (int i = threadIdx.x; i < 2 * kMoeCtas; i += kRouterThreads) p.arrivals[i] = 0;
    }
    f32x2 acc[NE][NT];
#pragma unroll
    for (int i = 0; i < NE; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = 0;
    for (int v = sub * 32 + lane; v < vecs; v += split * 32) {
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
    float hi[NE * NT], lo[NE * NT];
#pragma unroll
    for (int i = 0; i < NE * NT; ++i) {
        float b;
        a2av::split(acc[i / NT][i % NT], hi[i], b);
        lo[i] = 0.0f;
        two_sum(hi[i], lo[i], b, 0.0f);
    }
    warp_sums(hi, lo, lane);
    constexpr int kPer = 32 / (NE * NT);  // lanes that hold a value
    if (lane % kPer == 0) sums[warp][lane / kPer] = make_float2(hi[0], lo[0]);
    __syncthreads();
    if (sub == 0 && lane < NE * NT) {
        const int i = lane / NT, j = lane % NT;
        float h = 0.0f, l = 0.0f;
        for (int w = warp; w < warp + split; ++w) two_sum(h, l, sums[w][lane].x, sums[w][lane].y);
        if (e0 + i < p.E && t0 + j < p.T)
            p.logits[(t0 + j) * p.E + e0 + i] = fabsf(h) < __uint_as_float(0x7f800000u) ? h + l : h;
    }
}

template <bool BF16, bool R32>
cudaError_t launch_type(const MoeRouterLaunch &p, cudaStream_t stream) {
    const bool one = p.T <= 1;  // (without a token: nothing but the status)
    const int tiles = p.T == 0 ? 1 : one ? p.E : (p.E + 3) / 4 * ((p.T + 3) / 4);
    // Warps of a tile: so many that every SM has a block's.
    int split = kRouterWarps;
    while (split > 1 && tiles * split > kMoeCtas * kRouterWarps) split /= 2;
    const dim3 grid((tiles * split + kRouterWarps - 1) / kRouterWarps);
    return one ? launch_pdl(moe_router_kernel<BF16, R32, 1, 1>, grid, kRouterThreads, 0, 0, stream, p, split)
               : launch_pdl(moe_router_kernel<BF16, R32, 4, 4>, grid, kRouterThreads, 0, 0, stream, p, split);
}

// The choice, a warp a token: for more tokens than a CTA has warps (64 tokens over
// 256 experts, one after the other in every CTA, would take 18 us).
__global__ void __launch_bounds__(32) moe_choose_kernel(const MoeChoice c) {
    __shared__ float logits[kMoeExperts];
    const int t = blockIdx.x, lane = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    for (int e = lane; e < c.E; e += 32) logits[e] = __ldcg(c.logits + t * c.E + e);
    __syncwarp();
    int expert;
    float weight;
    moe_choose(c, logits, lane, expert, weight);
    if (lane < c.K) {
        const int pair = t * c.K + lane;
        c.chosen[pair] = make_int2(expert, __float_as_int(weight));
        if (c.experts) c.experts[pair] = expert;
        if (c.weights) c.weights[pair] = weight;
    }
}

}  // namespace

cudaError_t launch_moe_choose(const MoeChoice &c, cudaStream_t stream) {
    return launch_pdl(moe_choose_kernel, dim3(c.T), 32, 0, 0, stream, c);
}

cudaError_t launch_moe_router(const MoeRouterLaunch &p, bool bf16, bool router32, cudaStream_t stream) {
    if (router32) return bf16 ? launch_type<true, true>(p, stream) : launch_type<false, true>(p, stream);
    return bf16 ? launch_type<true, false>(p, stream) : launch_type<false, false>(p, stream);
}

}  // namespace a2av
