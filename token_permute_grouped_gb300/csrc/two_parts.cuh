// A value as two summands of a 16-bit type, for products whose other factor the
// tensor cores take in that type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace a2av {

// v as two summands of the element type that both have its sign (h toward zero,
// never all of v): the products of an infinity with them are infinities of one
// sign, as its product with v is, and not a NaN.  Values below the type's
// smallest are taken for it.
template <bool BF16>
__device__ __forceinline__ void two_parts(float v, uint32_t &h, uint32_t &l) {
    const auto value = [](uint32_t b) {
        if constexpr (BF16) return __uint_as_float(b << 16);
        else return __half2float(__ushort_as_half(static_cast<uint16_t>(b)));
    };
    if constexpr (BF16) h = __bfloat16_as_ushort(__float2bfloat16_rz(v));
    else h = __half_as_ushort(__float2half_rz(v));
    if (value(h) == v && (h & 0x7fffu) > 1) --h;  // the next value toward zero
    const float rest = v - value(h);
    if constexpr (BF16) l = __bfloat16_as_ushort(__float2bfloat16_rn(rest));
    else l = __half_as_ushort(__float2half_rn(rest));
    if ((l & 0x7fffu) == 0 && v != 0.0f) l = (h & 0x8000u) | 1u;
}
}  // namespace a2av
