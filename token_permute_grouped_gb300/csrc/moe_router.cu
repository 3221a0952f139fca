// The router of the expert layer for a few tokens: the logits l[t][e] = sum over h
// of x[t][h] router[e][h], and the choice of experts from them.
//
// A warp holds four experts' and four tokens' rows (one and one for a single
// token) against each other, or a part of them: `split` warps of a block take
// vectors of 8 along H in turn.  Their fp32 sums are joined with the rounding
// errors carried along, since a logit's last digits may decide a choice.  Bound by
// latency for few tokens, by the reads of the rows from L2 for many.
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

// A float as an integer of the same order; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t moe_order(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    if (v != v) return 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One warp chooses a token's experts from its logits: lane l looks after experts
// l, l + 32, ..., in descending order, and the lanes' first ones are compared K
// times.  Lane k < K has the k-th choice and its weight.
__device__ __forceinline__ void moe_choose(const MoeChoice &c, const float *logits, int lane, int &expert, float &weight) {
    constexpr int N = kMoeExperts / 32;
    const float low = -__uint_as_float(0x7f800000u);
    float l[N];
    float top = low;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        l[i] = lane + 32 * i < c.E ? logits[lane + 32 * i] : low;
        top = fmaxf(top, l[i]);
    }
    float total = 1.0f;
    if (c.score == A2AV_SCORE_SOFTMAX) {
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < c.E) total += expf(l[i] - top);
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    }
    const auto score = [&](float v) {
        return c.score == A2AV_SCORE_SOFTMAX ? expf(v - top) / total : 1.0f / (1.0f + expf(-v));
    };
    // A key (0: no expert; what is there is above, since the order of a NaN is 0 and
    // that of an infinity below the largest integer), and the logit's number.
    uint32_t key[N];
    int at[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        at[i] = i;
        key[i] = e < c.E ? moe_order(c.bias ? score(l[i]) + __ldg(c.bias + e) : l[i]) + 1 : 0;
    }
    // Insertion by neighbours: descending, equal keys stay in the experts' order.
#pragma unroll
    for (int pass = 1; pass < N; ++pass) {
        if (32 * pass >= c.E) break;
#pragma unroll
        for (int i = pass; i > 0; --i) {
            if (key[i] > key[i - 1]) {
                const uint32_t k = key[i];
                const int n = at[i];
                key[i] = key[i - 1], at[i] = at[i - 1];
                key[i - 1] = k, at[i - 1] = n;
            }
        }
    }
    float logit = 0.0f;
    expert = 0;
    for (int k = 0; k < c.K; ++k) {
        const uint32_t most = __reduce_max_sync(0xffffffffu, key[0]);
        const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, key[0] == most ? lane + 32 * at[0] : 0x7fffffff));
        if (lane == k) expert = e;
        if (lane == e % 32) {
#pragma unroll
            for (int i = 1; i < N; ++i) key[i - 1] = key[i], at[i - 1] = at[i];
            key[N - 1] = 0;
        }
    }
    // (The logit again, from where it was read.)
    if (lane < c.K) logit = logits[expert];
    float mine = lane < c.K ? score(logit) : 0.0f;
    if (c.renormalise) {
        // Of the scores only their ratios are left, taken relative to the largest chosen
        // logit m: all of them may lie below fp32's range (sigmoid below -88; softmax where
        // the bias chose), and their sum would be 0.  sigmoid(v) = e^v / (1 + e^v).
        float m = lane < c.K ? logit : low;
        for (int off = 4; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        float ratio = expf(logit - m);
        if (c.score == A2AV_SCORE_SOFTMAX) ratio = total == total ? ratio : total;  // (a NaN or +infinity among all logits)
        else ratio = m < 0.0f ? ratio / (1.0f + expf(logit)) : mine;
        if (lane < c.K) mine = ratio;
    }
    float sum = mine;
    for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    weight = (c.renormalise ? mine / sum : mine) * c.scale;
}

// The choice, a warp a token.  (In the products' CTAs, each for itself, it took as
// long for one token, and 18 us for 64 over 256 experts.)
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
