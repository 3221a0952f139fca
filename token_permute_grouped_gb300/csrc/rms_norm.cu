// RMS norm with the residual's addition and an 8-bit output, and its gradient.
//
//   s = x + residual, rstd = 1 / sqrt(mean(s^2) + eps), y = s rstd gamma
//   dx = dh + rstd (a - n mean(a n)),  a = dy gamma,  n = h rstd;  dgamma = sum dy n
//
// HBM-bound, one pass: a row (up to 65,528 values) stays in the registers of
// one block between the sum and the scaling, so each input is read once.
// Lanes hold 16-byte vectors of 8 values, neighbours next to each other, so
// that loads are coalesced and a scale block is 4 or 16 neighbouring lanes.
#include <algorithm>

#include "activation.cuh"
#include "ffn.h"
#include "quantise.cuh"

namespace a2av {

namespace {

__device__ __forceinline__ uint4 ld_once(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Sum over the block, the same in every thread.  `slots` alternates between
// two sets of 32 floats so that one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float v, float *slots) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
    if (warps == 1) return v;
    if (lane == 0) slots[threadIdx.x / 32] = v;
    __syncthreads();
    v = lane < warps ? slots[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// VPT: vectors of 8 values a thread holds.  MODE: a2av_qmode or kQuantNone.
template <bool BF16, int VPT, int MODE>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const RmsNormLaunch p) {
    __shared__ float slots[2][32];
    const int vecs = p.H / 8, T = blockDim.x, t = threadIdx.x;
    const uint4 *gamma = static_cast<const uint4 *>(p.gamma);
    int flip = 0;
    for (int row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + row * p.x_stride);
        const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.residual) + row * p.r_stride);
        const size_t out0 = static_cast<size_t>(row) * vecs;
        uint4 raw[VPT], res[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if (t + k * T < vecs) raw[k] = ld_once(x + t + k * T);
        if (p.residual) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (t + k * T < vecs) res[k] = ld_once(r + t + k * T);
        }
        float s[VPT][8];
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (t + k * T < vecs) {
                unpack8<BF16>(raw[k], s[k]);
                if (p.residual) {
                    float f[8];
                    unpack8<BF16>(res[k], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[k][i] += f[i];
                }
                if (p.h) static_cast<uint4 *>(p.h)[out0 + t + k * T] = pack8<BF16>(s[k]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += s[k][i] * s[k][i];
        }
        sum = block_sum(sum, slots[flip]);
        const float rstd = rsqrtf(sum / static_cast<float>(p.H) + p.eps);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        if (MODE == kQuantNone && !p.y) continue;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
            float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (v < vecs) {
                float g[8];
                unpack8<BF16>(__ldg(gamma + v), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = s[k][i] * rstd * g[i];
                if (p.y) static_cast<uint4 *>(p.y)[out0 + v] = pack8<BF16>(y);
            }
            if constexpr (MODE != kQuantNone) {
                uint8_t e8m0 = 0;
                float scale = 0.0f;
                const uint2 c = quantise8<MODE>(y, p.qtype, &e8m0, &scale);
                if (v < vecs) {
                    reinterpret_cast<uint2 *>(p.codes)[out0 + v] = c;
                    constexpr int kLanes = MODE == A2AV_QMODE_MX ? 4 : 16;
                    if (v % kLanes == 0) {
                        if constexpr (MODE == A2AV_QMODE_MX)
                            static_cast<uint8_t *>(p.scales)[(out0 + v) / kLanes] = e8m0;
                        else
                            static_cast<float *>(p.scales)[(out0 + v) / kLanes] = scale;
                    }
                }
            }
        }
    }
}

template <bool BF16, int VPT>
cudaError_t launch_norm_vpt(const RmsNormLaunch &p, int qmode, int threads, int grid, cudaStream_t stream) {
    if (qmode == kQuantNone) rms_norm_kernel<BF16, VPT, kQuantNone><<<grid, threads, 0, stream>>>(p);
    else if (qmode == A2AV_QMODE_MX) rms_norm_kernel<BF16, VPT, A2AV_QMODE_MX><<<grid, threads, 0, stream>>>(p);
    else rms_norm_kernel<BF16, VPT, A2AV_QMODE_GROUP128><<<grid, threads, 0, stream>>>(p);
    return cudaGetLastError();
}

// Threads for `vecs` vectors at VPT each: whole warps.
int threads_for(int vecs, int vpt) { return ((vecs + vpt - 1) / vpt + 31) / 32 * 32; }

// A block walks rows, keeping its share of dgamma in registers; the shares go
// to partial[block] and a second kernel adds them in block order.
template <bool BF16, int VPT>
__global__ void __launch_bounds__(1024) rms_norm_grad_kernel(const RmsNormGradLaunch p) {
    __shared__ float slots[2][32];
    const int vecs = p.H / 8, T = blockDim.x, t = threadIdx.x;
    const uint4 *gamma = static_cast<const uint4 *>(p.gamma);
    float dg[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[k][i] = 0.0f;
    int flip = 0;
    for (int row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
        const size_t r0 = static_cast<size_t>(row) * vecs;
        const uint4 *dy = static_cast<const uint4 *>(p.dy) + r0, *h = static_cast<const uint4 *>(p.h) + r0;
        const float rstd = __ldg(p.rstd + row);
        uint4 a[VPT], n[VPT], d[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
            a[k] = n[k] = d[k] = make_uint4(0, 0, 0, 0);
            if (v < vecs) {
                a[k] = ld_once(dy + v);
                n[k] = ld_once(h + v);
                if (p.dh) d[k] = ld_once(static_cast<const uint4 *>(p.dh) + r0 + v);
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
            if (v < vecs) {
                float fa[8], fn[8], g[8];
                unpack8<BF16>(a[k], fa);
                unpack8<BF16>(n[k], fn);
                unpack8<BF16>(__ldg(gamma + v), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = fa[i] * (fn[i] * rstd);
                    dg[k][i] += u;
                    dot += u * g[i];
                }
            }
        }
        dot = block_sum(dot, slots[flip]) / static_cast<float>(p.H);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
            if (v < vecs) {
                float fa[8], fn[8], g[8], o[8];
                unpack8<BF16>(a[k], fa);
                unpack8<BF16>(n[k], fn);
                unpack8<BF16>(__ldg(gamma + v), g);
                unpack8<BF16>(d[k], o);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += rstd * (fa[i] * g[i] - fn[i] * rstd * dot);
                static_cast<uint4 *>(p.dx)[r0 + v] = pack8<BF16>(o);
            }
        }
    }
    if (!p.dgamma) return;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = t + k * T;
        if (v < vecs) {
            float4 *out = reinterpret_cast<float4 *>(p.partial + static_cast<size_t>(blockIdx.x) * p.H) + 2 * v;
            out[0] = make_float4(dg[k][0], dg[k][1], dg[k][2], dg[k][3]);
            out[1] = make_float4(dg[k][4], dg[k][5], dg[k][6], dg[k][7]);
        }
    }
}

// dgamma[c] = sum over blocks of partial[block][c]: 32 columns a block of 32
// row slices, each slice in block order, the slices joined in order.
constexpr int kSlices = 16;
__global__ void __launch_bounds__(32 * kSlices) dgamma_sum_kernel(const float *__restrict__ partial, int blocks, int H,
                                                                  float *__restrict__ dgamma) {
    __shared__ float s[kSlices][33];
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (c < H)
        for (int b = slice; b < blocks; b += kSlices) sum += partial[static_cast<size_t>(b) * H + c];
    s[slice][lane] = sum;
    __syncthreads();
    if (slice == 0 && c < H) {
        for (int k = 1; k < kSlices; ++k) sum += s[k][lane];
        dgamma[c] = sum;
    }
}

constexpr int kGradBlocks = 608;

}  // namespace

cudaError_t launch_rms_norm(const RmsNormLaunch &p, bool bf16, int qmode, int sms, cudaStream_t stream) {
    const int vecs = p.H / 8;
    int vpt = 1;
    while (vpt < 8 && (threads_for(vecs, vpt) > 1024 || (p.rows > sms && vpt < 4))) vpt *= 2;
    const int threads = threads_for(vecs, vpt);
    const int grid = std::min(p.rows, sms * 16);
    switch (vpt) {
#define A2AV_NORM(V)                                                                       \
    return bf16 ? launch_norm_vpt<true, V>(p, qmode, threads, grid, stream)                \
                : launch_norm_vpt<false, V>(p, qmode, threads, grid, stream)
        case 1: A2AV_NORM(1);
        case 2: A2AV_NORM(2);
        case 4: A2AV_NORM(4);
        default: A2AV_NORM(8);
#undef A2AV_NORM
    }
}

int rms_norm_grad_blocks(int64_t rows, int64_t) { return static_cast<int>(std::min<int64_t>(rows, kGradBlocks)); }

cudaError_t launch_rms_norm_grad(const RmsNormGradLaunch &p, bool bf16, cudaStream_t stream) {
    const int vecs = p.H / 8;
    int vpt = 2;
    while (vpt < 8 && threads_for(vecs, vpt) > 1024) vpt *= 2;
    const int threads = threads_for(vecs, vpt);
    if (p.blocks > 0) {
        switch (vpt) {
#define A2AV_GRAD(V)                                                                                   \
    if (bf16) rms_norm_grad_kernel<true, V><<<p.blocks, threads, 0, stream>>>(p);                      \
    else rms_norm_grad_kernel<false, V><<<p.blocks, threads, 0, stream>>>(p);                          \
    break
            case 2: A2AV_GRAD(2);
            case 4: A2AV_GRAD(4);
            default: A2AV_GRAD(8);
#undef A2AV_GRAD
        }
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    if (p.dgamma)
        dgamma_sum_kernel<<<(p.H + 31) / 32, 32 * kSlices, 0, stream>>>(p.partial, p.blocks, p.H, p.dgamma);
    return cudaGetLastError();
}

}  // namespace a2av
