// Shared by the norms over rows (rms_norm.cu, layer_norm.cu): loads of values
// that are read once, sums over a row's threads, the reciprocal root.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace a2av {

__device__ __forceinline__ uint4 ld_once(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Sum over a row's threads, the same in every thread.  `slots` alternates
// between two sets so that one barrier a sum is enough; `bar` is the named
// barrier of the row's threads.  Partial sums are added with the rounding
// error carried along (two-sum), which leaves the error of the threads' own
// short sums, averaged over the row.
__device__ __forceinline__ void two_sum(float &hi, float &lo, float b_hi, float b_lo) {
    const float s = hi + b_hi, z = s - hi;
    lo += b_lo + ((hi - (s - z)) + (b_hi - z));
    hi = s;
}

__device__ __forceinline__ float2 row_sum(float v, float2 *slots, int t, int threads, int bar) {
    float lo = 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        two_sum(v, lo, __shfl_xor_sync(0xffffffffu, v, off), __shfl_xor_sync(0xffffffffu, lo, off));
    const int warps = threads / 32, lane = t % 32;
    if (warps > 1) {
        if (lane == 0) slots[t / 32] = make_float2(v, lo);
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
        const float2 w = lane < warps ? slots[lane] : make_float2(0.0f, 0.0f);
        v = w.x;
        lo = w.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            two_sum(v, lo, __shfl_xor_sync(0xffffffffu, v, off), __shfl_xor_sync(0xffffffffu, lo, off));
    }
    return make_float2(v, fabsf(v) < __uint_as_float(0x7f800000u) ? lo : 0.0f);  // (an infinite sum's error is a NaN)
}

// 1 / sqrt(sum / H + eps) for a sum of two parts: one Newton step on the
// hardware's reciprocal root, and in `lo` what is missing from it, the roundings
// of the mean among it.
__device__ __forceinline__ float inv_rms(float2 sum, float H, float eps, float &lo) {
    const float q = sum.x / H, q_lo = (fmaf(-q, H, sum.x) + sum.y) / H;
    const float v = q + eps, z = v - q;
    const float v_lo = (q - (v - z)) + (eps - z) + q_lo;
    float r = rsqrtf(v);
    lo = 0.0f;
    if (v > 0.0f && v < __uint_as_float(0x7f800000u)) {
        r = fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
        const float w = v * r, e = fmaf(v, r, -w);  // v r^2 = (w + e) r
        lo = -0.5f * r * (fmaf(w, r, -1.0f) + (e + v_lo * r) * r);
    }
    return r;
}

// Threads for `vecs` vectors at VPT each: whole warps.
inline int threads_for(int vecs, int vpt) { return ((vecs + vpt - 1) / vpt + 31) / 32 * 32; }

}  // namespace a2av
