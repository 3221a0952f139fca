// The work that follows from the choice of experts.
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

// By the whole block, of at least kMoeExperts threads; R rows a unit.
__device__ __forceinline__ void moe_plan(const MoeChoice &c, MoePlan &plan, int R) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    if (tid < kMoeExperts) plan.mask[tid] = 0;
    __syncthreads();
    for (int p = tid; p < c.T * c.K; p += blockDim.x) {
        const int2 v = __ldcg(c.chosen + p);
        plan.chosen[p] = static_cast<uint16_t>(v.x);
        plan.weight[p] = __int_as_float(v.y);
        atomicOr(&plan.mask[v.x], 1ull << (p / c.K));
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
