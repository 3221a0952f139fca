// 8-bit output with scales, shared by the kernels that end in one: E8M0
// scales per 32 values (mx) or float32 scales per 128 values (group128), in
// the formats the block-scaled product and the quantised reduce read.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

#include "a2av_quant_reduce.h"

namespace a2av {

constexpr int kQuantNone = -1;

// Largest exponent and largest finite value of a code format.
__device__ __forceinline__ int q_emax(int qtype) { return qtype == A2AV_Q_E4M3FN ? 8 : 15; }
__device__ __forceinline__ float q_max(int qtype) {
    return qtype == A2AV_Q_E4M3FN ? 448.0f : qtype == A2AV_Q_E5M2 ? 57344.0f : 127.0f;
}

__device__ __forceinline__ uint32_t fp8_pair(float a, float b, int qtype) {
    return qtype == A2AV_Q_E4M3FN ? __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)
                                  : __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
}

__device__ __forceinline__ uint32_t int8_code(float v) {
    return v == v ? static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(v, -127.0f), 127.0f))) & 0xffu : 0u;
}

// The codes of the 8 consecutive values y[] this lane holds, and their
// block's scale.  The lanes of a block are neighbours (4 lanes for mx, 16 for
// group128, starting at a multiple of that); every lane of the warp calls
// this, lanes without values with zeros.  The block's largest magnitude is
// taken over the bit patterns without their signs, in which an infinity is
// above every finite value and a NaN above that, so that neither is lost.
//
// mx: the scale is a power of two, so y * 2^-E is exact and the code is
// rounded once.  group128: one fp32 quotient qmax / m a block.
template <int MODE>
__device__ __forceinline__ uint2 quantise8(const float (&y)[8], int qtype, uint8_t *e8m0, float *scale) {
    constexpr int kLanes = MODE == A2AV_QMODE_MX ? 4 : 16;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    const bool finite = top < 0x7f800000u;
    float mult;
    if constexpr (MODE == A2AV_QMODE_MX) {
        // floor(log2) of a normal number is its exponent field less 127; of a
        // subnormal one (field 0) and of zero it is below the clamp.
        const int E = min(max(static_cast<int>(top >> 23) - 127 - q_emax(qtype), -127), 127);
        *e8m0 = finite ? static_cast<uint8_t>(E + 127) : 0xff;
        mult = finite ? __uint_as_float(static_cast<uint32_t>(127 - E) << 23) : __uint_as_float(0x7fc00000u);
    } else {
        const float m = fmaxf(__uint_as_float(top), 7.888609052210118e-31f);  // 2^-100
        *scale = finite ? m / q_max(qtype) : __uint_as_float(0x7fc00000u);
        mult = finite ? q_max(qtype) / m : __uint_as_float(0x7fc00000u);
    }
    uint32_t w[2];
    if (qtype == A2AV_Q_INT8) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = int8_code(y[4 * k] * mult) | int8_code(y[4 * k + 1] * mult) << 8 |
                   int8_code(y[4 * k + 2] * mult) << 16 | int8_code(y[4 * k + 3] * mult) << 24;
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = fp8_pair(y[4 * k] * mult, y[4 * k + 1] * mult, qtype) |
                   fp8_pair(y[4 * k + 2] * mult, y[4 * k + 3] * mult, qtype) << 16;
    }
    return make_uint2(w[0], w[1]);
}

}  // namespace a2av
