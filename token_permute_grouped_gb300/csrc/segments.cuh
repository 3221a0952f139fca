// The segment table of plan.cuh, faster where all (source, expert) counts fit
// one warp: a lane holds a count, and both prefix sums are shuffles.  It stands
// at the start of every kernel, where a call of a few microseconds feels it.
#pragma once

#include "plan.cuh"

namespace a2av {

// As build_segment_table; one full warp calls this.
__device__ __forceinline__ bool build_segments(const int32_t *__restrict__ recvCounts, int W, int e, int64_t A,
                                               SegmentTable &t, int lane) {
    const int E = W * e;
    if (E > 32) return build_segment_table(recvCounts, W, e, A, t, lane);
    const int32_t c = lane < E ? recvCounts[lane] : 0;  // segment (w, j) = (lane / e, lane % e)
    // Expert-major slot `lane` holds segment (w, j) = (lane % W, lane / W).
    const int32_t d = __shfl_sync(0xffffffffu, c, lane < E ? lane % W * e + lane / W : 0) * (lane < E ? 1 : 0);
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
    if (lane < E) {
        t.src[lane] = static_cast<int32_t>(src - c);
        t.dst[lane] = dst - d;
    }
    const int64_t total = __shfl_sync(0xffffffffu, src, 31);
    if (lane == 0) t.dst[E] = static_cast<int32_t>(total);
    const bool bad = __any_sync(0xffffffffu, c < 0);
    __syncwarp();
    return !bad && total == A;
}

}  // namespace a2av
