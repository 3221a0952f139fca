// 16-bit vectors as fp32, and the gated block's activations with their slopes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "a2av_ffn.h"

namespace a2av {

template <bool BF16>
__device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi) {
    if constexpr (BF16) {  // a bf16 is the upper half of the float of the same value
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        lo = f.x;
        hi = f.y;
    }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2f(float lo, float hi) {  // nearest even
    if constexpr (BF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    } else {
        __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    }
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    unpack2<BF16>(v.x, f[0], f[1]);
    unpack2<BF16>(v.y, f[2], f[3]);
    unpack2<BF16>(v.z, f[4], f[5]);
    unpack2<BF16>(v.w, f[6], f[7]);
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2f<BF16>(f[0], f[1]), pack2f<BF16>(f[2], f[3]), pack2f<BF16>(f[4], f[5]),
                      pack2f<BF16>(f[6], f[7]));
}

// 1 / (1 + e^-z).  The fast exponential and quotient are good to a few units
// in the last place of fp32, far below the rounding of any output; where
// 1 + e^-z passes 2^126 the quotient is 0 in place of a value below 2^-126.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// Both activations are g * sigmoid(z): z = g for silu; for gelu, since
// (1 + tanh(t)) / 2 = sigmoid(2t), z = 2 sqrt(2/pi) (g + 0.044715 g^3), which
// has no cancellation near g = 0.
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGelu3 = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    if constexpr (ACT == A2AV_ACT_SILU) return g * sigmoid(g);
    return g * sigmoid(kGelu2 * (g + kGelu3 * g * g * g));
}

// act(g) and its slope s + g z' s (1 - s), s = sigmoid(z).
template <int ACT>
__device__ __forceinline__ float act_value_slope(float g, float &slope) {
    if constexpr (ACT == A2AV_ACT_SILU) {
        const float s = sigmoid(g);
        slope = s + g * s * (1.0f - s);
        return g * s;
    }
    const float s = sigmoid(kGelu2 * (g + kGelu3 * g * g * g));
    slope = s + g * (kGelu2 * (1.0f + 3.0f * kGelu3 * g * g)) * (s * (1.0f - s));
    return g * s;
}

}  // namespace a2av
