// 8-bit output with scales, shared by the kernels that end in one: E8M0
// scales per 32 values (mx) or float32 scales per 128 values (group128), in
// the formats the block-scaled product and the quantised reduce read.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

#include "a2av_quant_reduce.h"
#include "activation.cuh"

namespace a2av {

// What a kernel's 8-bit output is, when compiling: none, or a mode with a type.
constexpr int kQuantNone = -1;
constexpr int quant_kind(int qmode, int qtype) { return qmode * 4 + qtype; }
template <int KIND>
struct Quant {
    static constexpr bool kAny = KIND != kQuantNone;
    static constexpr bool kMx = KIND / 4 == A2AV_QMODE_MX;
    static constexpr int kType = KIND % 4;
    static constexpr int kLanes = kMx ? 4 : 16;  // neighbouring lanes of a scale block
    static constexpr int kEmax = kType == A2AV_Q_E4M3FN ? 8 : 15;
    static constexpr float kMax = kType == A2AV_Q_E4M3FN ? 448.0f : kType == A2AV_Q_E5M2 ? 57344.0f : 127.0f;
};

// Four values as codes, the first in the low byte.
template <int QT>
__device__ __forceinline__ uint32_t codes4(f32x2 p, f32x2 q) {
    float a, b, c, d;
    split(p, a, b);
    split(q, c, d);
    if constexpr (QT == A2AV_Q_INT8) {
        // A scaled magnitude is at most 127 (1 + 2^-22), so no value rounds past 127; a NaN becomes 0.
        return (static_cast<uint32_t>(__float2int_rn(a)) & 0xffu) | (static_cast<uint32_t>(__float2int_rn(b)) & 0xffu) << 8 |
               (static_cast<uint32_t>(__float2int_rn(c)) & 0xffu) << 16 | static_cast<uint32_t>(__float2int_rn(d)) << 24;
    } else {
        constexpr __nv_fp8_interpretation_t kind = QT == A2AV_Q_E4M3FN ? __NV_E4M3 : __NV_E5M2;
        return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, kind)) |
               static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, kind)) << 16;
    }
}

// Largest magnitude of three; a NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Codes and scales of K vectors of 8 values y[k][] that this lane holds; the
// lanes of a scale block are neighbours, starting at a multiple of kLanes.
// Every lane of the warp calls this, lanes without values with zeros.
// store(k, codes, e8m0, scale) takes the results.
//
// mx: the scale is a power of two, so y * 2^-E is exact and the code is
// rounded once.  E steps where the block's largest magnitude passes a power of
// two, so a y that is one rounding off there would halve or double a whole
// block's scale.  Within 8 units of y's last place of a power of two (a few
// blocks in a million) reaches(k, pw) decides, from more than fp32, whether
// one of this lane's magnitudes is at least pw.
// The norm's y is always that near.  An activation of a far negative gate may be
// up to 54 units off, but every product of 16-bit factors that comes near a power
// of two was tried (some hundred mantissa pairs an activation), and none beyond
// these 8 units falls on the wrong side of it.
// UNITS: those 8, or what a caller's y needs.
// group128: one fp32 quotient qmax / m a block.
template <int KIND, int K, uint32_t UNITS = 8, typename Reaches, typename Store>
__device__ __forceinline__ void quantise(const f32x2 (&y)[K][4], Reaches reaches, Store store) {
    using Q = Quant<KIND>;
    uint32_t top[K];
    bool near = false;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) split(y[k][i], v[2 * i], v[2 * i + 1]);
        float m = max3_abs(max3_abs(v[0], v[1], v[2]), v[3], max3_abs(v[4], v[5], max3_abs(v[6], v[7], 0.0f)));
#pragma unroll
        for (int off = 1; off < Q::kLanes; off <<= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, m, off);
            m = max3_abs(m, o, 0.0f);
        }
        top[k] = __float_as_uint(m) & 0x7fffffffu;  // infinity above every finite value, NaN above that
        near |= ((top[k] + UNITS) & 0x7fffffu) < 2 * UNITS && top[k] - 0x00800001u < 0x7f000000u;  // normal numbers only
    }
    int step[K];
#pragma unroll
    for (int k = 0; k < K; ++k) step[k] = 0;
    if constexpr (Q::kMx) {
        if (__any_sync(0xffffffffu, near)) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const bool here = ((top[k] + UNITS) & 0x7fffffu) < 2 * UNITS && top[k] - 0x00800001u < 0x7f000000u;
                const uint32_t pw = (top[k] + UNITS) & 0x7f800000u;
                int hit = here && reaches(k, __uint_as_float(pw)) ? 1 : 0;
#pragma unroll
                for (int off = 1; off < Q::kLanes; off <<= 1) hit |= __shfl_xor_sync(0xffffffffu, hit, off);
                // the exponent of pw if it is reached, else the one below, against what the fp32 value says
                if (here) step[k] = static_cast<int>(pw >> 23) - 1 + hit - static_cast<int>(top[k] >> 23);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const bool finite = top[k] < 0x7f800000u;
        float mult, scale = 0.0f;
        uint8_t e8m0 = 0;
        if constexpr (Q::kMx) {
            // floor(log2) of a normal number is its exponent field less 127; of a
            // subnormal one (field 0) and of zero it is below the clamp.
            const int E = max(static_cast<int>(top[k] >> 23) + step[k] - Q::kEmax, 0);  // E + 127, at most 254
            e8m0 = finite ? static_cast<uint8_t>(E) : 0xff;
            mult = __uint_as_float(finite ? static_cast<uint32_t>(254 - E) << 23 : 0x7fc00000u);
        } else {
            const float m = fmaxf(__uint_as_float(top[k]), 7.888609052210118e-31f);  // 2^-100
            scale = finite ? m * (1.0f / Q::kMax) : __uint_as_float(0x7fc00000u);
            mult = finite ? Q::kMax / m : __uint_as_float(0x7fc00000u);
        }
        const f32x2 m2 = both(mult);
        store(k,
              make_uint2(codes4<Q::kType>(mul2(y[k][0], m2), mul2(y[k][1], m2)),
                         codes4<Q::kType>(mul2(y[k][2], m2), mul2(y[k][3], m2))),
              e8m0, scale);
    }
}

}  // namespace a2av
