// The gated activation with an 8-bit output, and the gated block's
// element-wise gradient.  Both are HBM-bound single passes.
//
//   v = act(gate) up -> T and / or codes with scales
//   dG = dh U act'(G),  dU = dh act(G)
#include <algorithm>

#include "activation.cuh"
#include "ffn.h"
#include "quantise.cuh"

namespace a2av {

namespace {

constexpr int kGluThreads = 256;
constexpr int kGluVecs = 4;  // vectors a thread has in flight

// A thread takes vectors of 8 columns, kGluThreads apart, in the order of the
// output.  N is a whole number of scale blocks, so a block never spans rows
// and its lanes are neighbours here too.
template <bool BF16, int ACT, int MODE>
__global__ void __launch_bounds__(kGluThreads) glu_quant_kernel(const GluLaunch p) {
    const int vpr = p.N / 8;
    const int64_t total = p.rows * vpr;
    const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kGluThreads * kGluVecs) + threadIdx.x;
    uint4 g[kGluVecs], u[kGluVecs];
#pragma unroll
    for (int k = 0; k < kGluVecs; ++k) {
        const int64_t v = v0 + k * kGluThreads;
        g[k] = u[k] = make_uint4(0, 0, 0, 0);
        if (v < total) {
            const int64_t row = v / vpr, off = row * p.stride + (v - row * vpr) * 8;
            g[k] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.gate) + off));
            u[k] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.up) + off));
        }
    }
#pragma unroll
    for (int k = 0; k < kGluVecs; ++k) {
        const int64_t v = v0 + k * kGluThreads;
        float fg[8], fu[8];
        unpack8<BF16>(g[k], fg);
        unpack8<BF16>(u[k], fu);
#pragma unroll
        for (int i = 0; i < 8; ++i) fg[i] = act_value<ACT>(fg[i]) * fu[i];
        if (p.h && v < total) static_cast<uint4 *>(p.h)[v] = pack8<BF16>(fg);
        if constexpr (MODE != kQuantNone) {
            uint8_t e8m0 = 0;
            float scale = 0.0f;
            const uint2 c = quantise8<MODE>(fg, p.qtype, &e8m0, &scale);
            if (v < total) {
                reinterpret_cast<uint2 *>(p.codes)[v] = c;
                constexpr int kLanes = MODE == A2AV_QMODE_MX ? 4 : 16;
                if (v % kLanes == 0) {
                    if constexpr (MODE == A2AV_QMODE_MX) static_cast<uint8_t *>(p.scales)[v / kLanes] = e8m0;
                    else static_cast<float *>(p.scales)[v / kLanes] = scale;
                }
            }
        }
    }
}

template <bool BF16, int ACT>
__global__ void __launch_bounds__(kGluThreads) glu_grad_kernel(const GluGradLaunch p) {
    const int64_t vecs = p.n / 8;
    for (int64_t v = static_cast<int64_t>(blockIdx.x) * kGluThreads + threadIdx.x; v < vecs;
         v += static_cast<int64_t>(gridDim.x) * kGluThreads) {
        const uint4 d = __ldcs(static_cast<const uint4 *>(p.dh) + v);
        const float4 g0 = __ldcs(reinterpret_cast<const float4 *>(p.gate) + 2 * v);
        const float4 g1 = __ldcs(reinterpret_cast<const float4 *>(p.gate) + 2 * v + 1);
        const float4 u0 = __ldcs(reinterpret_cast<const float4 *>(p.up) + 2 * v);
        const float4 u1 = __ldcs(reinterpret_cast<const float4 *>(p.up) + 2 * v + 1);
        const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
        const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
        float fd[8], dg[8], du[8];
        unpack8<BF16>(d, fd);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float slope;
            const float a = act_value_slope<ACT>(g[i], slope);
            dg[i] = fd[i] * u[i] * slope;
            du[i] = fd[i] * a;
        }
        static_cast<uint4 *>(p.dgate)[v] = pack8<BF16>(dg);
        static_cast<uint4 *>(p.dup)[v] = pack8<BF16>(du);
    }
}

template <bool BF16, int ACT>
cudaError_t launch_glu_mode(const GluLaunch &p, int qmode, int64_t grid, cudaStream_t stream) {
    const unsigned g = static_cast<unsigned>(grid);
    if (qmode == kQuantNone) glu_quant_kernel<BF16, ACT, kQuantNone><<<g, kGluThreads, 0, stream>>>(p);
    else if (qmode == A2AV_QMODE_MX) glu_quant_kernel<BF16, ACT, A2AV_QMODE_MX><<<g, kGluThreads, 0, stream>>>(p);
    else glu_quant_kernel<BF16, ACT, A2AV_QMODE_GROUP128><<<g, kGluThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_glu_quant(const GluLaunch &p, bool bf16, int act, int qmode, int, cudaStream_t stream) {
    const int64_t vecs = p.rows * (p.N / 8);
    // At most 2^31 / 8 * 65528 / 1024 blocks, below the grid limit of 2^31 - 1 for every allowed shape
    // that fits the card's memory.
    const int64_t grid = (vecs + kGluThreads * kGluVecs - 1) / (kGluThreads * kGluVecs);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (bf16)
        return act == A2AV_ACT_SILU ? launch_glu_mode<true, A2AV_ACT_SILU>(p, qmode, grid, stream)
                                    : launch_glu_mode<true, A2AV_ACT_GELU_TANH>(p, qmode, grid, stream);
    return act == A2AV_ACT_SILU ? launch_glu_mode<false, A2AV_ACT_SILU>(p, qmode, grid, stream)
                                : launch_glu_mode<false, A2AV_ACT_GELU_TANH>(p, qmode, grid, stream);
}

cudaError_t launch_glu_grad(const GluGradLaunch &p, bool bf16, int act, int sms, cudaStream_t stream) {
    const int64_t blocks = (p.n / 8 + kGluThreads - 1) / kGluThreads;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(sms) * 8));
    if (bf16) {
        if (act == A2AV_ACT_SILU) glu_grad_kernel<true, A2AV_ACT_SILU><<<grid, kGluThreads, 0, stream>>>(p);
        else glu_grad_kernel<true, A2AV_ACT_GELU_TANH><<<grid, kGluThreads, 0, stream>>>(p);
    } else {
        if (act == A2AV_ACT_SILU) glu_grad_kernel<false, A2AV_ACT_SILU><<<grid, kGluThreads, 0, stream>>>(p);
        else glu_grad_kernel<false, A2AV_ACT_GELU_TANH><<<grid, kGluThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace a2av
