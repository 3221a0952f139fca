// The gated activation with an 8-bit output, v = act(gate) up -> T and / or
// codes with scales: one HBM-bound pass.
#include "activation.cuh"
#include "ffn.h"
#include "pdl.cuh"
#include "quantise.cuh"

namespace a2av {

namespace {

// 128 threads of two vectors each, eight blocks an SM: measured on 34,502 rows
// of 2 x 2048 bf16 columns to E4M3FN codes, 60.2 us (5.9 TB/s, 87 % of the
// copy rate); 256 threads 72.2, four vectors a thread 68.9, one 83.8 (too few
// bytes in flight), more resident blocks spill (72.0 with ten).
constexpr int kGluThreads = 128;
constexpr int kGluVecs = 2;  // vectors a thread has in flight
constexpr int kGluBlocks = 8;

// Whether one of the 8 products' magnitudes is at least pw, in double and out
// of line: for the few blocks next to a power of two.
template <bool BF16, int ACT>
__device__ __noinline__ bool glu_reaches(uint4 g, uint4 u, float pw) {
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
    bool hit = false;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        float a[2], b[2];
        split(unpack2<BF16>(gw[i]), a[0], a[1]);
        split(unpack2<BF16>(uw[i]), b[0], b[1]);
#pragma unroll 1
        for (int j = 0; j < 2; ++j)
            hit |= fabs(act_value_wide<ACT>(j ? a[1] : a[0]) * static_cast<double>(j ? b[1] : b[0])) >= pw;
    }
    return hit;
}

// A thread takes vectors of 8 columns, kGluThreads apart, in the order of the
// output.  N is a whole number of scale blocks, so a block never spans rows
// and its lanes are neighbours here too.  The row of a vector comes from
// products with 1 / (N / 8) (64 bits once a block, 32 bits inside it); both
// are exact for every allowed size.
template <bool BF16, int ACT, int KIND>
__global__ void __launch_bounds__(kGluThreads, kGluBlocks) glu_quant_kernel(const GluLaunch p) {
    using Q = Quant<KIND>;
    const uint32_t vpr = p.N / 8;
    const int64_t total = p.rows * vpr;
    const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kGluThreads * kGluVecs);
    const int64_t row0 = vpr == 1 ? v0 : static_cast<int64_t>(__umul64hi(v0, p.inv64));
    const uint32_t c0 = static_cast<uint32_t>(v0 - row0 * vpr) + threadIdx.x;
    uint4 g[kGluVecs], u[kGluVecs];
    pdl_trigger();
    pdl_wait();
#pragma unroll
    for (int k = 0; k < kGluVecs; ++k) {
        g[k] = u[k] = make_uint4(0, 0, 0, 0);
        if (v0 + threadIdx.x + k * kGluThreads < total) {
            const uint32_t c = c0 + k * kGluThreads, r = vpr == 1 ? c : __umulhi(c, p.inv32);
            const int64_t off = (row0 + r) * p.stride + (c - r * vpr) * 8;
            g[k] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.gate) + off));
            u[k] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.up) + off));
        }
    }
    f32x2 y[kGluVecs][4];
#pragma unroll
    for (int k = 0; k < kGluVecs; ++k) {
        f32x2 fg[4], fu[4];
        unpack8<BF16>(g[k], fg);
        unpack8<BF16>(u[k], fu);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[k][i] = mul2(act_value<ACT>(fg[i]), fu[i]);
        const int64_t v = v0 + threadIdx.x + k * kGluThreads;
        if (p.h && v < total) static_cast<uint4 *>(p.h)[v] = pack8<BF16>(y[k]);
    }
    if constexpr (Q::kAny) {
        quantise<KIND, kGluVecs>(
            y, [&](int k, float pw) { return glu_reaches<BF16, ACT>(g[k], u[k], pw); },
            [&](int k, uint2 codes, uint8_t e8m0, float scale) {
                const int64_t v = v0 + threadIdx.x + k * kGluThreads;
                if (v >= total) return;
                reinterpret_cast<uint2 *>(p.codes)[v] = codes;
                if (v % Q::kLanes == 0) {
                    if constexpr (Q::kMx) static_cast<uint8_t *>(p.scales)[v / Q::kLanes] = e8m0;
                    else static_cast<float *>(p.scales)[v / Q::kLanes] = scale;
                }
            });
    }
}

template <bool BF16, int ACT>
cudaError_t launch_glu_kind(const GluLaunch &p, int kind, unsigned grid, cudaStream_t stream) {
    switch (kind) {
#define A2AV_KIND(...)                                                                      \
    case __VA_ARGS__:                                                                       \
        return launch_pdl(glu_quant_kernel<BF16, ACT, __VA_ARGS__>, grid, kGluThreads, 0, 0, stream, p)
        A2AV_KIND(kQuantNone);
        A2AV_KIND(quant_kind(A2AV_QMODE_MX, A2AV_Q_E4M3FN));
        A2AV_KIND(quant_kind(A2AV_QMODE_MX, A2AV_Q_E5M2));
        A2AV_KIND(quant_kind(A2AV_QMODE_GROUP128, A2AV_Q_E4M3FN));
        A2AV_KIND(quant_kind(A2AV_QMODE_GROUP128, A2AV_Q_E5M2));
        A2AV_KIND(quant_kind(A2AV_QMODE_GROUP128, A2AV_Q_INT8));
#undef A2AV_KIND
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_glu_quant(GluLaunch p, bool bf16, int act, int kind, cudaStream_t stream) {
    const int64_t vecs = p.rows * (p.N / 8);
    const int64_t grid = (vecs + kGluThreads * kGluVecs - 1) / (kGluThreads * kGluVecs);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;  // more than 8 TB of rows
    p.inv64 = UINT64_MAX / (p.N / 8) + 1;
    p.inv32 = UINT32_MAX / (p.N / 8) + 1;
    const unsigned g = static_cast<unsigned>(grid);
    if (bf16)
        return act == A2AV_ACT_SILU ? launch_glu_kind<true, A2AV_ACT_SILU>(p, kind, g, stream)
                                    : launch_glu_kind<true, A2AV_ACT_GELU_TANH>(p, kind, g, stream);
    return act == A2AV_ACT_SILU ? launch_glu_kind<false, A2AV_ACT_SILU>(p, kind, g, stream)
                                : launch_glu_kind<false, A2AV_ACT_GELU_TANH>(p, kind, g, stream);
}

}  // namespace a2av
