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
#include "pdl.cuh"
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

// VPT: vectors of 8 values a thread holds.  KIND: the 8-bit output.  MAXT:
// threads at most.  A block that walks several rows requests the next one's
// values before it reduces the current row (up to two vectors a thread; more
// would not leave registers for it).
template <bool BF16, int VPT, int KIND, int MAXT>
__global__ void __launch_bounds__(MAXT) rms_norm_kernel(const RmsNormLaunch p) {
    using Q = Quant<KIND>;
    constexpr bool PRE = VPT <= 2;
    __shared__ float2 slots[2][32];
    const int vecs = p.H / 8, T = blockDim.x, t = threadIdx.x;
    const uint4 *gamma = static_cast<const uint4 *>(p.gamma);
    uint4 raw[VPT], res[VPT];
    const auto load = [&](int row) {
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + row * p.x_stride);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if (t + k * T < vecs) raw[k] = ld_once(x + t + k * T);
        if (p.residual) {
            const uint4 *r =
                reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.residual) + row * p.r_stride);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (t + k * T < vecs) res[k] = ld_once(r + t + k * T);
        }
    };
    int flip = 0;
    const int step = gridDim.x;
    const int last = p.rows - step;  // rows below it have a next one (row + step may not fit an int)
    pdl_trigger();
    pdl_wait();
    if (PRE) load(blockIdx.x);
    for (int row = blockIdx.x; row < p.rows; row = row < last ? row + step : p.rows, flip ^= 1) {
        const size_t out0 = static_cast<size_t>(row) * vecs;
        if (!PRE) load(row);
        f32x2 s[VPT][4];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[k][i] = 0;
            if (t + k * T < vecs) {
                unpack8<BF16>(raw[k], s[k]);
                if (p.residual) {
                    f32x2 f[4];
                    unpack8<BF16>(res[k], f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[k][i] = add2(s[k][i], f[i]);
                }
            }
        }
        if (PRE && row < last) load(row + step);
        f32x2 sum2 = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (p.h && t + k * T < vecs) static_cast<uint4 *>(p.h)[out0 + t + k * T] = pack8<BF16>(s[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum2 = fma2(s[k][i], s[k][i], sum2);
        }
        float sum, odd;
        split(sum2, sum, odd);
        const float2 total = row_sum(sum + odd, slots[flip], t, T, 0);
        float rstd_lo;
        const float rstd = inv_rms(total, static_cast<float>(p.H), p.eps, rstd_lo);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        if (!Q::kAny && !p.y) continue;
        f32x2 y[VPT][4];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[k][i] = 0;
            if (v < vecs) {
                f32x2 g[4];
                unpack8<BF16>(__ldg(gamma + v), g);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[k][i] = mul2(mul2(s[k][i], both(rstd)), g[i]);
                if (p.y) static_cast<uint4 *>(p.y)[out0 + v] = pack8<BF16>(y[k]);
            }
        }
        if constexpr (Q::kAny) {
            // y's two roundings and rstd's, each with its error: |y| - pw is
            // exact for the values in question.
            const auto reaches = [&](int k, float pw) {
                const int v = t + k * T;
                if (v >= vecs) return false;
                f32x2 g2[4];
                unpack8<BF16>(__ldg(gamma + v), g2);
                bool hit = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a[2], g[2], z[2];
                    split(s[k][i], a[0], a[1]);
                    split(g2[i], g[0], g[1]);
                    split(y[k][i], z[0], z[1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float q = a[j] * rstd, r = fmaf(a[j], rstd, -q);
                        const float err = fmaf(q, g[j], -z[j]) + (r + a[j] * rstd_lo) * g[j];
                        hit |= fabsf(z[j]) - pw + copysignf(1.0f, z[j]) * err >= 0.0f;
                    }
                }
                return hit;
            };
            quantise<KIND, VPT>(y, reaches, [&](int k, uint2 codes, uint8_t e8m0, float scale) {
                const int v = t + k * T;
                if (v >= vecs) return;
                reinterpret_cast<uint2 *>(p.codes)[out0 + v] = codes;
                if (v % Q::kLanes == 0) {
                    if constexpr (Q::kMx) static_cast<uint8_t *>(p.scales)[(out0 + v) / Q::kLanes] = e8m0;
                    else static_cast<float *>(p.scales)[(out0 + v) / Q::kLanes] = scale;
                }
            });
        }
    }
}

template <bool BF16, int VPT, int MAXT>
cudaError_t launch_norm_vpt(const RmsNormLaunch &p, int kind, int threads, int grid, cudaStream_t stream) {
    switch (kind) {
#define A2AV_KIND(...)                                                                             \
    case __VA_ARGS__:                                                                              \
        return launch_pdl(rms_norm_kernel<BF16, VPT, __VA_ARGS__, MAXT>, grid, threads, 0, 0, stream, p)
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

// Threads for `vecs` vectors at VPT each: whole warps.
int threads_for(int vecs, int vpt) { return ((vecs + vpt - 1) / vpt + 31) / 32 * 32; }

// A block holds R rows at a time (blockDim = T x R), each walked on by its own
// T threads, which keep their share of dgamma in registers; at the end the
// block adds its rows' shares in order and stores one row of partial sums, and
// a second kernel adds those in block order.
template <bool BF16, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) rms_norm_grad_kernel(const RmsNormGradLaunch p) {
    constexpr bool PRE = VPT <= 2;
    __shared__ float2 slots[2][32];
    extern __shared__ float4 share[];
    const int vecs = p.H / 8, T = blockDim.x, t = threadIdx.x, R = blockDim.y, g = threadIdx.y;
    const uint4 *gamma = static_cast<const uint4 *>(p.gamma);
    f32x2 dg[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[k][i] = 0;
    uint4 a[VPT], n[VPT], d[VPT], na[VPT], nn[VPT], nd[VPT];  // dy, h, dh of this row and of the next
    float rstd = 0.0f, nrstd = 0.0f;
    const auto load = [&](int row, uint4 (&ra)[VPT], uint4 (&rn)[VPT], uint4 (&rd)[VPT], float &rs) {
        const size_t r0 = static_cast<size_t>(row) * vecs;
        rs = __ldg(p.rstd + row);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
            if (v < vecs) {
                ra[k] = ld_once(static_cast<const uint4 *>(p.dy) + r0 + v);
                rn[k] = ld_once(static_cast<const uint4 *>(p.h) + r0 + v);
                if (p.dh) rd[k] = ld_once(static_cast<const uint4 *>(p.dh) + r0 + v);
            }
        }
    };
    int flip = 0;
    const int step = gridDim.x * R, last = p.rows - step;  // as above
    int row = blockIdx.x * R + g;
    pdl_wait();
    if (PRE && row < p.rows) load(row, na, nn, nd, nrstd);
    for (; row < p.rows; row = row < last ? row + step : p.rows, flip ^= 1) {
        const size_t r0 = static_cast<size_t>(row) * vecs;
        if (PRE) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) a[k] = na[k], n[k] = nn[k], d[k] = nd[k];
            rstd = nrstd;
            if (row < last) load(row + step, na, nn, nd, nrstd);
        } else {
            load(row, a, n, d, rstd);
        }
        f32x2 dot2 = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
            if (v < vecs) {
                f32x2 fa[4], fn[4], gm[4];
                unpack8<BF16>(a[k], fa);
                unpack8<BF16>(n[k], fn);
                unpack8<BF16>(__ldg(gamma + v), gm);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x2 u = mul2(fa[i], mul2(fn[i], both(rstd)));
                    dg[k][i] = add2(dg[k][i], u);
                    dot2 = fma2(u, gm[i], dot2);
                }
            }
        }
        float dot, odd;
        split(dot2, dot, odd);
        const float2 total = row_sum(dot + odd, slots[flip] + g * (T / 32), t, T, 1 + g);
        // dx = dh + rstd (a - n m), in this order: n and m are of the values' own size
        // for every scale of the row, while rstd^2 may be out of range.
        const float m = (total.x + total.y) / static_cast<float>(p.H);
        const f32x2 r2 = both(rstd), m2 = both(-m);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
            if (v < vecs) {
                f32x2 fa[4], fn[4], gm[4], o[4] = {0, 0, 0, 0};
                unpack8<BF16>(a[k], fa);
                unpack8<BF16>(n[k], fn);
                unpack8<BF16>(__ldg(gamma + v), gm);
                if (p.dh) unpack8<BF16>(d[k], o);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = fma2(fma2(mul2(fn[i], r2), m2, mul2(fa[i], gm[i])), r2, o[i]);
                static_cast<uint4 *>(p.dx)[r0 + v] = pack8<BF16>(o);
            }
        }
    }
    pdl_trigger();  // the sum over the blocks may be launched; it waits for this grid's end
    if (!p.dgamma) return;
    float4 *out = reinterpret_cast<float4 *>(p.blocks == 1 ? p.dgamma : p.partial + static_cast<size_t>(blockIdx.x) * p.H);
    for (int turn = 0; turn < R; ++turn) {
        if (turn == g) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = t + k * T;
                if (v < vecs) {
                    float4 lo, hi;
                    split(dg[k][0], lo.x, lo.y);
                    split(dg[k][1], lo.z, lo.w);
                    split(dg[k][2], hi.x, hi.y);
                    split(dg[k][3], hi.z, hi.w);
                    if (turn > 0) {
                        const float4 l = share[2 * v], h = share[2 * v + 1];
                        lo = make_float4(l.x + lo.x, l.y + lo.y, l.z + lo.z, l.w + lo.w);
                        hi = make_float4(h.x + hi.x, h.y + hi.y, h.z + hi.z, h.w + hi.w);
                    }
                    float4 *to = turn == R - 1 ? out : share;
                    to[2 * v] = lo;
                    to[2 * v + 1] = hi;
                }
            }
        }
        __syncthreads();
    }
}

// dgamma[c] = sum over blocks of partial[block][c]: 32 columns a block of
// kSlices slices of the partial sums, each in block order, the slices joined in
// order: the same sum every time.  About 3 us behind the kernel above (8192 rows of
// 7168: 88.4 us together, 91.8 with 16 slices, 99 with 8).
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) dgamma_sum_kernel(const float *__restrict__ partial, int blocks, int H,
                                                                  float *__restrict__ dgamma) {
    __shared__ float s[kSlices][33];
    pdl_trigger();
    pdl_wait();  // the partial sums are visible
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

// One block of 512 threads an SM, with the next row's three vectors requested
// while a row is reduced: 16,384 x 2048 bf16 rows take 46 us with the sum over
// the blocks (5.8 TB/s, 86 % of the copy rate; 40.5 without it, 6.6 TB/s), two
// blocks without the early request 52, two of 256 threads with it 51 (and twice
// the partial sums).
constexpr int kGradBlocks = 152;
constexpr int kGradThreads = 512;

// Resident threads an SM that the norm's grid is made for: its 64 registers a
// thread allow 1024.  Two vectors a thread: 12,288 x 7168 bf16 rows to E4M3FN
// codes take 96 us (6.4 TB/s, 95 % of the copy rate); without the next row's
// early request 118, four vectors 104, one 127.
constexpr int kNormThreadsPerSm = 1024;

struct GradShape {
    int vpt, threads, rows;  // vectors a thread, threads a row, rows a block
};
GradShape grad_shape(int64_t H) {
    const int vecs = static_cast<int>(H / 8);
    int vpt = 2;
    while (vpt < 8 && threads_for(vecs, vpt) > (vpt == 2 ? 512 : 1024)) vpt *= 2;
    const int threads = threads_for(vecs, vpt);
    // (the shares of dgamma of a block with several rows meet in at most 32 KB)
    return {vpt, threads, std::max(1, std::min(kGradThreads / threads, 8))};
}

template <bool BF16>
cudaError_t launch_norm_type(const RmsNormLaunch &p, int kind, int sms, cudaStream_t stream) {
    const int vecs = p.H / 8;
    const auto go = [&](auto launch, int vpt) {
        const int threads = threads_for(vecs, vpt);
        return launch(p, kind, threads, std::min(p.rows, sms * std::max(1, kNormThreadsPerSm / threads)), stream);
    };
    // A vector a thread where an SM has one row at most, and no next row's values to
    // hold (us, one / two vectors: 1 row of 2048 1.9 / 2.2, 152 rows 2.2 / 2.6; 152
    // of 7168 3.1 / 3.1, 304 of 7168 4.8 / 4.0, 608 of 2048 3.1 / 3.1).
    if (p.rows <= sms && vecs <= 1024) return go(launch_norm_vpt<BF16, 1, 1024>, 1);
    if (vecs <= 2048) return go(launch_norm_vpt<BF16, 2, 1024>, 2);
    if (vecs <= 4096) return go(launch_norm_vpt<BF16, 4, 1024>, 4);
    return go(launch_norm_vpt<BF16, 8, 1024>, 8);
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormLaunch &p, bool bf16, int kind, int sms, cudaStream_t stream) {
    return bf16 ? launch_norm_type<true>(p, kind, sms, stream) : launch_norm_type<false>(p, kind, sms, stream);
}

int rms_norm_grad_blocks(int64_t rows, int64_t H) {
    // Up to two turns of its rows by one block, whose sum is then all of it.
    const int64_t r = grad_shape(H).rows;
    return rows <= 2 * r ? static_cast<int>(std::min<int64_t>(rows, 1))
                         : static_cast<int>(std::min<int64_t>((rows + r - 1) / r, kGradBlocks));
}

cudaError_t launch_rms_norm_grad(const RmsNormGradLaunch &p, bool bf16, cudaStream_t stream) {
    const GradShape shape = grad_shape(p.H);
    if (p.blocks > 0) {
        const dim3 block(shape.threads, shape.rows);
        const size_t smem = shape.rows > 1 ? static_cast<size_t>(p.H) * 4 : 0;
        cudaError_t err;
        switch (shape.vpt) {
#define A2AV_GRAD(V, MAXT)                                                                             \
    err = bf16 ? launch_pdl(rms_norm_grad_kernel<true, V, MAXT>, p.blocks, block, smem, 0, stream, p)  \
               : launch_pdl(rms_norm_grad_kernel<false, V, MAXT>, p.blocks, block, smem, 0, stream, p); \
    break
            case 2: A2AV_GRAD(2, 512);
            case 4: A2AV_GRAD(4, 1024);
            default: A2AV_GRAD(8, 1024);
#undef A2AV_GRAD
        }
        if (err != cudaSuccess) return err;
    }
    if (!p.dgamma || p.blocks == 1) return cudaSuccess;
    return launch_pdl(dgamma_sum_kernel, (p.H + 31) / 32, 32 * kSlices, 0, 0, stream,
                      static_cast<const float *>(p.partial), p.blocks, p.H, p.dgamma);
}

}  // namespace a2av
