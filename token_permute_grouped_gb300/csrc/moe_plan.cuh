// The choice of experts, and the work that follows from it.
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
    const float mine = lane < c.K ? score(logit) : 0.0f;
    float sum = mine;
    for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    weight = (c.renormalise ? mine / sum : mine) * c.scale;
}

// By the whole block, of at least kMoeExperts threads; R rows a unit.  The choice
// is made here, by a warp a token, from logits in shared memory (store: and given
// out), or read where c.chosen has it.
__device__ __forceinline__ void moe_plan(const MoeChoice &c, MoePlan &plan, const float *logits, int R, bool store) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, nwarps = blockDim.x / 32;
    if (tid < kMoeExperts) plan.mask[tid] = 0;
    __syncthreads();
    if (c.chosen) {
        for (int p = tid; p < c.T * c.K; p += blockDim.x) {
            const int2 v = __ldcg(c.chosen + p);
            plan.chosen[p] = static_cast<uint16_t>(v.x);
            plan.weight[p] = __int_as_float(v.y);
            atomicOr(&plan.mask[v.x], 1ull << (p / c.K));
        }
    } else {
        for (int t = warp; t < c.T; t += nwarps) {
            int expert;
            float weight;
            moe_choose(c, logits + t * c.E, lane, expert, weight);
            if (lane < c.K) {
                const int pair = t * c.K + lane;
                plan.chosen[pair] = static_cast<uint16_t>(expert);
                plan.weight[pair] = weight;
                atomicOr(&plan.mask[expert], 1ull << t);
                if (store && c.experts) c.experts[pair] = expert;
                if (store && c.weights) c.weights[pair] = weight;
            }
        }
    }
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
