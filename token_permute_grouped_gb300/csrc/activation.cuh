// 16-bit vectors as fp32 pairs, and the gated block's activations with their
// slopes.
//
// Two fp32 values share a 64-bit register and one instruction for each product
// or sum (mul / add / fma .f32x2: each half rounded like the scalar one).  The
// element-wise kernels and the GEMM epilogues that use these would otherwise be
// bound by instruction issue, not by memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "a2av_ffn.h"

namespace a2av {

using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair_of(float lo, float hi) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void split(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 both(float v) { return pair_of(v, v); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

template <bool BF16>
__device__ __forceinline__ f32x2 unpack2(uint32_t w) {
    if constexpr (BF16) {  // a bf16 is the upper half of the float of the same value
        return pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        return pair_of(f.x, f.y);
    }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(f32x2 v) {  // nearest even
    float lo, hi;
    split(v, lo, hi);
    if constexpr (BF16) {
        __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&b);
    } else {
        __half2 b = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&b);
    }
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &v, f32x2 (&f)[4]) {
    f[0] = unpack2<BF16>(v.x);
    f[1] = unpack2<BF16>(v.y);
    f[2] = unpack2<BF16>(v.z);
    f[3] = unpack2<BF16>(v.w);
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const f32x2 (&f)[4]) {
    return make_uint4(pack2<BF16>(f[0]), pack2<BF16>(f[1]), pack2<BF16>(f[2]), pack2<BF16>(f[3]));
}

// 1 / (1 + e^-z).  The hardware's exponential and reciprocal are good to a few
// units in the last place of fp32, far below the rounding of any output; where
// 1 + e^-z passes 2^126 the quotient is 0 in place of a value below 2^-126.
__device__ __forceinline__ f32x2 sigmoid2(f32x2 z) {
    float a, b;
    split(mul2(z, both(-1.4426950408889634f)), a, b);  // -log2(e)
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    split(add2(pair_of(a, b), both(1.0f)), a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return pair_of(a, b);
}

// Both activations are g * sigmoid(z): z = g for silu; for gelu, since
// (1 + tanh(t)) / 2 = sigmoid(2t), z = 2 sqrt(2/pi) (g + 0.044715 g^3), which
// has no cancellation near g = 0.
constexpr float kGelu1 = 1.5957691216057308f;             // 2 sqrt(2/pi)
constexpr float kGelu3 = 1.5957691216057308f * 0.044715f;  // its product with 0.044715

template <int ACT>
__device__ __forceinline__ f32x2 act_value(f32x2 g) {
    if constexpr (ACT == A2AV_ACT_SILU) return mul2(g, sigmoid2(g));
    const f32x2 z = mul2(g, fma2(mul2(g, g), both(kGelu3), both(kGelu1)));
    return mul2(g, sigmoid2(z));
}

// act(g) in double, out of line: for the few values next to a power of two.
template <int ACT>
__device__ __noinline__ double act_value_wide(double g) {
    const double z = ACT == A2AV_ACT_SILU ? g : 2.0 * 0.7978845608028654 * (g + 0.044715 * g * g * g);
    return g / (1.0 + exp(-z));
}

// act(g) and its slope s + g z' s (1 - s), s = sigmoid(z).
template <int ACT>
__device__ __forceinline__ f32x2 act_value_slope(f32x2 g, f32x2 &slope) {
    f32x2 z = g, gdz = g;
    if constexpr (ACT != A2AV_ACT_SILU) {
        z = mul2(g, fma2(mul2(g, g), both(kGelu3), both(kGelu1)));
        // Beyond |g| of 16, s (1 - s) is 0 in fp32, and so is its product with g z',
        // which is not left to grow out of range.
        float lo, hi;
        split(g, lo, hi);
        const f32x2 c = pair_of(fminf(fmaxf(lo, -16.0f), 16.0f), fminf(fmaxf(hi, -16.0f), 16.0f));
        gdz = mul2(c, fma2(mul2(c, c), both(3.0f * kGelu3), both(kGelu1)));
    }
    const f32x2 s = sigmoid2(z);
    const f32x2 rest = fma2(s, both(-1.0f), both(1.0f));
    slope = fma2(gdz, mul2(s, rest), s);
    return mul2(g, s);
}

}  // namespace a2av
