// The choice of experts, made from the logits by every block that needs it (a
// few tokens: cheaper than handing it on), and the work that follows from it.
#pragma once

#include <cstdint>

#include "moe.h"
#include "ptx.cuh"

namespace a2av {

// A unit is up to R rows of one expert: (token, slot) pairs, listed expert after
// expert, an expert's tokens ascending.
struct MoeUnit {
    uint16_t expert, first, rows;  // first: of its pairs
};

struct MoePlan {
    unsigned long long mask[kMoeExperts];  // tokens that chose an expert
    uint16_t chosen[kMoeTokens * kMoeChosen];
    float weight[kMoeTokens * kMoeChosen];  // by pair t * K + k
    uint16_t pairs[kMoeTokens * kMoeChosen];
    MoeUnit unit[kMoeTokens * kMoeChosen];
    uint16_t start[kMoeExperts];  // first pair of an expert
    int32_t row_sums[kMoeExperts / 32], unit_sums[kMoeExperts / 32];
    int32_t units;
};

// A float as an integer of the same order; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t moe_order(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    if (v != v) return 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One warp chooses token t's experts: lane l looks after experts l, l + 32, ...
__device__ __forceinline__ void moe_choose(const MoeChoice &c, MoePlan &plan, int t, int lane, bool store) {
    constexpr int N = kMoeExperts / 32;
    float l[N];
    float top = -__uint_as_float(0x7f800000u);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < c.E ? __ldcg(c.logits + t * c.E + e) : -__uint_as_float(0x7f800000u);
        top = fmaxf(top, l[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float total = 1.0f;
    if (c.score == A2AV_SCORE_SOFTMAX) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < c.E) total += expf(l[i] - top);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    }
    const auto score = [&](float v) {
        return c.score == A2AV_SCORE_SOFTMAX ? expf(v - top) / total : 1.0f / (1.0f + expf(-v));
    };
    uint32_t key[N];  // 0: not there, or chosen already; what is there is above
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0;
        // (the order of a NaN is 0 and that of an infinity below the largest integer, so 1 more is never 0)
        if (e < c.E) key[i] = moe_order(c.bias ? score(l[i]) + __ldg(c.bias + e) : l[i]) + 1;
    }
    float mine = 0.0f;  // lane k: the k-th score
    int expert = 0;
    for (int k = 0; k < c.K; ++k) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, best == most ? lane + 32 * at : 0x7fffffff));
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i == e) key[i] = 0, v = l[i];
        v = __shfl_sync(0xffffffffu, v, e % 32);
        if (lane == k) mine = score(v), expert = e;
    }
    float sum = lane < c.K ? mine : 0.0f;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane < c.K) {
        const float w = (c.renormalise ? mine / sum : mine) * c.scale;
        const int pair = t * c.K + lane;
        plan.chosen[pair] = static_cast<uint16_t>(expert);
        plan.weight[pair] = w;
        atomicOr(&plan.mask[expert], 1ull << t);
        if (store && c.experts) c.experts[pair] = expert;
        if (store && c.weights) c.weights[pair] = w;
    }
}

// By the whole block, of at least kMoeExperts threads; R rows a unit.
__device__ __forceinline__ void moe_plan(const MoeChoice &c, MoePlan &plan, int R, bool store) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, nwarps = blockDim.x / 32;
    if (tid < kMoeExperts) plan.mask[tid] = 0;
    __syncthreads();
    for (int t = warp; t < c.T; t += nwarps) moe_choose(c, plan, t, lane, store);
    __syncthreads();
    const int rows = tid < kMoeExperts ? __popcll(plan.mask[tid]) : 0;
    const int units = (rows + R - 1) / R;
    int row_inc = rows, unit_inc = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, row_inc, off), b = __shfl_up_sync(0xffffffffu, unit_inc, off);
        if (lane >= off) row_inc += a, unit_inc += b;
    }
    if (tid < kMoeExperts && lane == 31) plan.row_sums[warp] = row_inc, plan.unit_sums[warp] = unit_inc;
    __syncthreads();
    if (tid < kMoeExperts) {
        int row0 = row_inc - rows, unit0 = unit_inc - units;
        for (int w = 0; w < warp; ++w) row0 += plan.row_sums[w], unit0 += plan.unit_sums[w];
        plan.start[tid] = static_cast<uint16_t>(row0);
        for (int i = 0; i < units; ++i)
            plan.unit[unit0 + i] = MoeUnit{static_cast<uint16_t>(tid), static_cast<uint16_t>(row0 + i * R),
                                           static_cast<uint16_t>(min(R, rows - i * R))};
        if (tid == kMoeExperts - 1) plan.units = unit0 + units;
    }
    __syncthreads();
    for (int p = tid; p < c.T * c.K; p += blockDim.x) {
        const int e = plan.chosen[p], t = p / c.K;
        plan.pairs[plan.start[e] + __popcll(plan.mask[e] & ((1ull << t) - 1))] = static_cast<uint16_t>(p);
    }
    __syncthreads();
}

}  // namespace a2av
