// Layer norm with the residual's addition and an 8-bit output, and its gradient.
//
//   s = x + residual, mu = mean(s), rstd = 1 / sqrt(mean((s - mu)^2) + eps)
//   y = (s - mu) rstd gamma + beta
//   dx = dh + rstd (a - mean(a) - n mean(a n)),  a = dy gamma,  n = (h - mu) rstd
//   dgamma = sum dy n,  dbeta = sum dy
//
// HBM-bound, one pass, laid out as the RMS norm (rms_norm.cu): a row stays in
// the registers of one block between its sums and the scaling, the next row's
// values are requested before the current one is reduced.  Values and squares are
// summed in one reduction; where the mean is more than half of the deviation, the
// squares are summed again about a short value next to the mean, from what the
// registers hold, so that a row's offset costs no digits.  With codes the instructions count as much as HBM:
// gamma and beta wait in shared memory as fp32 (109 us against 115.6 for mx codes).
// 12,288 x 7168 bf16 rows with a residual: to mx codes 106 us, to codes per 128 99
// (6.2 TB/s, 93% of a copy's rate; 127 with a reduction a sum in every row); in rows
// that are summed again 137 and 122.  Without a residual, 43% of the bytes, 94 and 86:
// bound by the instructions.  Above 16,384 values a row, four or eight vectors a thread,
// registers are spilled: 2048 x 20,480 to codes per 128 97, 1024 x 65,408 450 (40 and 70
// at a copy's rate).
#include <algorithm>

#include "activation.cuh"
#include "ffn.h"
#include "pair.cuh"
#include "pdl.cuh"
#include "quantise.cuh"
#include "rows.cuh"

namespace a2av {

namespace {

// y has three roundings and may lose a few digits against beta: its exponent is
// decided with its errors carried along within this many units of a power of two.
constexpr uint32_t kNearUnits = 64;

// Sums over a row's threads of two values, each in two parts, as row_sum; one
// barrier.  The lower half of a warp looks after the first value, the upper half
// after the second: half the instructions of two sums, which would be a third of
// the kernel's.
__device__ __forceinline__ void row_sums(float a, float b, float4 *slots, int t, int threads, float2 &sa, float2 &sb) {
    const int warps = threads / 32, lane = t % 32;
    const bool upper = lane >= 16;
    float v = upper ? b : a, lo = 0.0f;
    two_sum(v, lo, __shfl_xor_sync(0xffffffffu, upper ? a : b, 16), 0.0f);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
        two_sum(v, lo, __shfl_xor_sync(0xffffffffu, v, off), __shfl_xor_sync(0xffffffffu, lo, off));
    if (warps > 1) {
        float2 *const mine = reinterpret_cast<float2 *>(slots) + (upper ? 1 : 0);  // of warp w: at 2 w
        if (lane % 16 == 0) mine[2 * (t / 32)] = make_float2(v, lo);
        __syncthreads();
        const int w = lane % 16;
        const float2 x = w < warps ? mine[2 * w] : make_float2(0.0f, 0.0f);
        v = x.x, lo = x.y;
        if (warps > 16) {
            const float2 y = w + 16 < warps ? mine[2 * (w + 16)] : make_float2(0.0f, 0.0f);
            two_sum(v, lo, y.x, y.y);
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
            two_sum(v, lo, __shfl_xor_sync(0xffffffffu, v, off), __shfl_xor_sync(0xffffffffu, lo, off));
    }
    if (!(fabsf(v) < __uint_as_float(0x7f800000u))) lo = 0.0f;  // (an infinite sum's error is a NaN)
    sa = make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, lo, 0));
    sb = make_float2(__shfl_sync(0xffffffffu, v, 16), __shfl_sync(0xffffffffu, lo, 16));
}

// sum / H of a sum of two parts, in two parts; inv = 1 / H.
__device__ __forceinline__ float mean_of(float2 sum, float H, float inv, float &lo) {
    const float q = sum.x * inv;
    lo = (fmaf(-q, H, sum.x) + sum.y) * inv;
    return q;
}

// 1 / sqrt(v + eps) for a v of two parts: one Newton step on the hardware's
// reciprocal root, and in `lo` what is missing from it.
__device__ __forceinline__ float inv_root(float v_hi, float v_part, float eps, float &lo) {
    const float v = v_hi + eps, z = v - v_hi;
    const float v_lo = (v_hi - (v - z)) + (eps - z) + v_part;
    float r = rsqrtf(v);
    lo = 0.0f;
    if (v > 0.0f && v < __uint_as_float(0x7f800000u)) {
        r = fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
        const float w = v * r, e = fmaf(v, r, -w);  // v r^2 = (w + e) r
        lo = -0.5f * r * (fmaf(w, r, -1.0f) + (e + v_lo * r) * r);
    }
    return r;
}

// a + b, b of two 16-bit elements: one instruction each, without a conversion first
// (mx codes of 12,288 x 7168 118.5 -> 115.6 us; without codes HBM is the bound, and
// packed additions were 2% faster).
template <bool BF16>
__device__ __forceinline__ f32x2 add_elements(f32x2 a, uint32_t b) {
    float x, y;
    split(a, x, y);
    if constexpr (BF16)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
            : "+f"(x), "+f"(y)
            : "r"(b));
    else
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %1, h, %1;\n\t}"
            : "+f"(x), "+f"(y)
            : "r"(b));
    return pair_of(x, y);
}

// VPT: vectors of 8 values a thread holds.  KIND: the 8-bit output.
template <bool BF16, int VPT, int KIND>
__global__ void __launch_bounds__(1024) layer_norm_kernel(const LayerNormLaunch p) {
    using Q = Quant<KIND>;
    constexpr bool PRE = VPT <= 2, WIDE = VPT == 2 && Q::kAny;
    __shared__ float4 slots[2][32];  // of both sums, by row
    __shared__ float2 again[32];     // of the squares about the mean
    extern __shared__ float4 wide[];  // gamma and beta: four planes of a vector's values 0-3 and 4-7
    const int vecs = p.H / 8, T = blockDim.x, t = threadIdx.x;
    const uint4 *gamma = static_cast<const uint4 *>(p.gamma), *beta = static_cast<const uint4 *>(p.beta);
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
    const float H = static_cast<float>(p.H), inv = 1.0f / H;
    pdl_trigger();
    pdl_wait();
    if (PRE) load(blockIdx.x);
    if (WIDE) {  // (a thread reads what it has written)
        const auto put = [&](const uint4 *from, float4 *to, int v) {
            f32x2 f[4] = {0, 0, 0, 0};
            if (from) unpack8<BF16>(__ldg(from + v), f);
            split(f[0], to[v].x, to[v].y), split(f[1], to[v].z, to[v].w);
            split(f[2], to[vecs + v].x, to[vecs + v].y), split(f[3], to[vecs + v].z, to[vecs + v].w);
        };
        for (int v = t; v < vecs; v += T) {
            put(gamma, wide, v);
            put(beta, wide + 2 * vecs, v);
        }
    }
    const auto weights = [&](const uint4 *from, const float4 *in, int v, f32x2 (&f)[4]) {
        if (WIDE) {
            const float4 a = in[v], b = in[vecs + v];
            f[0] = pair_of(a.x, a.y), f[1] = pair_of(a.z, a.w), f[2] = pair_of(b.x, b.y), f[3] = pair_of(b.z, b.w);
        } else if (from) {
            unpack8<BF16>(__ldg(from + v), f);
        }
    };
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
                    if constexpr (Q::kAny) {
                        s[k][0] = add_elements<BF16>(s[k][0], res[k].x);
                        s[k][1] = add_elements<BF16>(s[k][1], res[k].y);
                        s[k][2] = add_elements<BF16>(s[k][2], res[k].z);
                        s[k][3] = add_elements<BF16>(s[k][3], res[k].w);
                    } else {
                        f32x2 f[4];
                        unpack8<BF16>(res[k], f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[k][i] = add2(s[k][i], f[i]);
                    }
                }
            }
        }
        if (PRE && row < last) load(row + step);
        f32x2 sum2 = 0, sq2 = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            sum2 = add2(sum2, add2(add2(s[k][0], s[k][1]), add2(s[k][2], s[k][3])));
#pragma unroll
            for (int i = 0; i < 4; ++i) sq2 = fma2(s[k][i], s[k][i], sq2);
        }
        if (p.h) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (t + k * T < vecs) static_cast<uint4 *>(p.h)[out0 + t + k * T] = pack8<BF16>(s[k]);
        }
        float sum, odd, sq, sq_odd;
        split(sum2, sum, odd);
        split(sq2, sq, sq_odd);
        float2 total, squares;
        row_sums(sum + odd, sq + sq_odd, slots[flip], t, T, total, squares);
        const float inf = __uint_as_float(0x7f800000u);
        float mu_lo, mu = mean_of(total, H, inv, mu_lo);
        if (!(fabsf(mu_lo) < inf)) mu_lo = 0.0f;  // (of an infinite sum)
        const float mean = mu;
        // The squares about the mean are those about 0 less H mu^2 = mu total, each in
        // two parts.  Where that is more than a quarter of what is left, or the squares
        // about 0 overflow, the values are taken about c, and the squares summed anew.  c
        // is the mean's first 12 bits: a 16-bit value's difference from it is exact, and
        // mu - c below a quarter of the deviation; or, where the mean is over 500 times the
        // deviation (or the squares about 0 overflow), the mean in fp32.
        const float m = mu * total.x, m_lo = fmaf(mu, total.x, -m) + (mu * total.y + mu_lo * total.x);
        const float left = squares.x - m;
        if (squares.x < inf && left > 4.0f * m) {
            two_sum(squares.x, squares.y, -m, -m_lo);
        } else {
            const uint32_t bits = squares.x < inf && left > 0x1p-18f * m ? 0xfffff000u : 0xffffffffu;
            const float c = __uint_as_float(__float_as_uint(mu) & bits);
            sq2 = 0;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (t + k * T < vecs) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[k][i] = add2(s[k][i], both(-c));
                        sq2 = fma2(s[k][i], s[k][i], sq2);
                    }
                }
            }
            mu = fabsf(mu) < inf ? mu - c : 0.0f;
            split(sq2, sq, sq_odd);
            squares = row_sum(sq + sq_odd, again, t, T, 0);
            const float d2 = mu * mu, e = H * d2;  // H (mu - c)^2, likewise (mu - c is of 12 bits, its square exact)
            if (e > 0.0f) two_sum(squares.x, squares.y, -e, -fmaf(2.0f * H * mu, mu_lo, fmaf(H, d2, -e)));
            if (squares.x < 0.0f) squares = make_float2(0.0f, 0.0f);
        }
        float var_lo, rstd_lo;
        const float var = mean_of(squares, H, inv, var_lo);
        const float rstd = inv_root(var, fabsf(var_lo) < inf ? var_lo : 0.0f, p.eps, rstd_lo);
        if (t == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        if (!Q::kAny && !p.y) continue;
        const f32x2 scale = both(rstd), shift = both(-fmaf(mu, rstd, mu_lo * rstd));  // (mu is below half of the deviation here)
        f32x2 y[VPT][4];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = t + k * T;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[k][i] = 0;
            if (v < vecs) {
                f32x2 g[4], b[4] = {0, 0, 0, 0};
                weights(gamma, wide, v, g);
                weights(beta, wide + 2 * vecs, v, b);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[k][i] = fma2(fma2(s[k][i], scale, shift), g[i], b[i]);
                if (p.y) static_cast<uint4 *>(p.y)[out0 + v] = pack8<BF16>(y[k]);
            }
        }
        if constexpr (Q::kAny) {
            // y's roundings and those of the mean and of rstd, each with its error: near pw,
            // the difference of the sum's head from it is exact.  (What stays are the roundings
            // of a thread's sums of values and squares.)
            const auto reaches = [&](int k, float pw) {
                const int v = t + k * T;
                if (v >= vecs) return false;
                f32x2 g2[4], b2[4] = {0, 0, 0, 0};
                unpack8<BF16>(__ldg(gamma + v), g2);
                if (beta) unpack8<BF16>(__ldg(beta + v), b2);
                bool hit = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a[2], g[2], b[2];
                    split(s[k][i], a[0], a[1]);
                    split(g2[i], g[0], g[1]);
                    split(b2[i], b[0], b[1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float d = a[j], rest = 0.0f;
                        two_sum(d, rest, -mu, -mu_lo);  // a - mu
                        const float n = d * rstd, n_lo = fmaf(d, rstd, -n) + (d * rstd_lo + rest * rstd);
                        float z = n * g[j], z_lo = fmaf(n, g[j], -z) + n_lo * g[j];
                        two_sum(z, z_lo, b[j], 0.0f);
                        hit |= fabsf(z) - pw + copysignf(1.0f, z) * z_lo >= 0.0f;
                    }
                }
                return hit;
            };
            quantise<KIND, VPT, kNearUnits>(y, reaches, [&](int k, uint2 codes, uint8_t e8m0, float scale) {
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

constexpr int kMaxWide = 16384 * 8;  // the widest row of two vectors a thread

template <bool BF16, int VPT>
cudaError_t launch_norm_vpt(const LayerNormLaunch &p, int kind, int threads, int grid, cudaStream_t stream) {
    const size_t smem = VPT == 2 && kind != kQuantNone ? static_cast<size_t>(p.H) * 8 : 0;
    const auto go = [&](auto kern) {
        if (smem > 48 * 1024) {
            const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxWide);
            if (err != cudaSuccess) return err;
        }
        return launch_pdl(kern, grid, threads, smem, 0, stream, p);
    };
    switch (kind) {
#define A2AV_KIND(...) \
    case __VA_ARGS__: return go(layer_norm_kernel<BF16, VPT, __VA_ARGS__>)
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

// Sums over a row's threads of two values; one barrier.
__device__ __forceinline__ float2 row_sum_two(float a, float b, float2 *slots, int t, int threads, int bar) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    const int warps = threads / 32, lane = t % 32;
    if (warps > 1) {
        if (lane == 0) slots[t / 32] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
        const float2 w = lane < warps ? slots[lane] : make_float2(0.0f, 0.0f);
        a = w.x, b = w.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, off);
            b += __shfl_xor_sync(0xffffffffu, b, off);
        }
    }
    return make_float2(a, b);
}

// A block holds R rows at a time (blockDim = T x R), each walked on by its own
// T threads, which keep their share of dgamma and dbeta in registers; at the end
// the block adds its rows' shares in order and stores one row of partial sums
// (dgamma's H, then dbeta's), and a second kernel adds those in block order.  The
// blocks of few rows are one cluster instead, each of which adds a part of the
// columns over all of them, in order, from their shared memory.
template <bool BF16, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) layer_norm_grad_kernel(const LayerNormGradLaunch p) {
    constexpr bool PRE = VPT <= 2;
    __shared__ float2 slots[2][32];
    extern __shared__ float4 share[];
    const int vecs = p.H / 8, T = blockDim.x, t = threadIdx.x, R = blockDim.y, g = threadIdx.y;
    const uint4 *gamma = static_cast<const uint4 *>(p.gamma);
    f32x2 dg[VPT][4], db[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[k][i] = db[k][i] = 0;
    uint4 a[VPT], n[VPT], d[VPT], na[VPT], nn[VPT], nd[VPT];  // dy, h, dh of this row and of the next
    float rstd = 0.0f, nrstd = 0.0f, mu = 0.0f, nmu = 0.0f;
    const auto load = [&](int row, uint4 (&ra)[VPT], uint4 (&rn)[VPT], uint4 (&rd)[VPT], float &rs, float &rm) {
        const size_t r0 = static_cast<size_t>(row) * vecs;
        rs = __ldg(p.rstd + row);
        rm = __ldg(p.mean + row);
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
    if (PRE && row < p.rows) load(row, na, nn, nd, nrstd, nmu);
    for (; row < p.rows; row = row < last ? row + step : p.rows, flip ^= 1) {
        const size_t r0 = static_cast<size_t>(row) * vecs;
        if (PRE) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) a[k] = na[k], n[k] = nn[k], d[k] = nd[k];
            rstd = nrstd, mu = nmu;
            if (row < last) load(row + step, na, nn, nd, nrstd, nmu);
        } else {
            load(row, a, n, d, rstd, mu);
        }
        const f32x2 r2 = both(rstd), mu2 = both(-mu);
        f32x2 sum2 = 0, dot2 = 0;
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
                    const f32x2 u = mul2(fa[i], mul2(add2(fn[i], mu2), r2));
                    dg[k][i] = add2(dg[k][i], u);
                    db[k][i] = add2(db[k][i], fa[i]);
                    dot2 = fma2(u, gm[i], dot2);
                    sum2 = fma2(fa[i], gm[i], sum2);
                }
            }
        }
        float sum, sum_odd, dot, dot_odd;
        split(sum2, sum, sum_odd);
        split(dot2, dot, dot_odd);
        const float2 total = row_sum_two(sum + sum_odd, dot + dot_odd, slots[flip] + g * (T / 32), t, T, 1 + g);
        // dx = dh + rstd (a - mean(a) - n m), in this order: n and m are of the values'
        // own size for every scale of the row, while rstd^2 may be out of range.
        const f32x2 ma2 = both(-total.x / static_cast<float>(p.H)), m2 = both(-total.y / static_cast<float>(p.H));
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
                for (int i = 0; i < 4; ++i)
                    o[i] = fma2(fma2(mul2(add2(fn[i], mu2), r2), m2, fma2(fa[i], gm[i], ma2)), r2, o[i]);
                static_cast<uint4 *>(p.dx)[r0 + v] = pack8<BF16>(o);
            }
        }
    }
    pdl_trigger();  // the sum over the blocks may be launched; it waits for this grid's end
    if (!p.dgamma) return;
    const bool alone = p.blocks == 1, joined = p.clustered && !alone;
    float *sums = p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.H;
    float4 *const outs[2] = {reinterpret_cast<float4 *>(alone ? p.dgamma : sums),
                             reinterpret_cast<float4 *>(alone ? p.dbeta : sums + p.H)};
    const auto put = [&](int turn, int v, const f32x2 (&s)[4], float4 *shared, float4 *out) {
        float4 lo, hi;
        split(s[0], lo.x, lo.y);
        split(s[1], lo.z, lo.w);
        split(s[2], hi.x, hi.y);
        split(s[3], hi.z, hi.w);
        if (turn > 0) {
            const float4 l = shared[2 * v], h = shared[2 * v + 1];
            lo = make_float4(l.x + lo.x, l.y + lo.y, l.z + lo.z, l.w + lo.w);
            hi = make_float4(h.x + hi.x, h.y + hi.y, h.z + hi.z, h.w + hi.w);
        }
        float4 *to = turn == R - 1 && !joined ? out : shared;
        to[2 * v] = lo;
        to[2 * v + 1] = hi;
    };
    for (int turn = 0; turn < R; ++turn) {
        if (turn == g) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = t + k * T;
                if (v < vecs) {
                    put(turn, v, dg[k], share, outs[0]);
                    put(turn, v, db[k], share + p.H / 4, outs[1]);
                }
            }
        }
        __syncthreads();
    }
    if (joined) {
        pair::sync_all();  // every block's sums are in its shared memory
        const int cols = 2 * p.H / 4;  // of 4 values: dgamma's, then dbeta's
        for (int c = blockIdx.x * T * R + g * T + t; c < cols; c += gridDim.x * T * R) {
            const uint32_t at = smem_u32(share + c);
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int b = 0; b < p.blocks; ++b) {
                float4 v;
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                             : "r"(pair::map_to_rank(at, b))
                             : "memory");
                sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
            }
            reinterpret_cast<float4 *>(c < cols / 2 ? p.dgamma : p.dbeta)[c < cols / 2 ? c : c - cols / 2] = sum;
        }
        pair::sync_all();  // no block leaves while another may read its sums
    }
}

// out[c] = sum over blocks of partial[block][c], c over dgamma's columns and then
// dbeta's: 32 columns a block of kSlices slices of the partial sums, each in
// block order, the slices joined in order: the same sums every time.
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) column_sums_kernel(const float *__restrict__ partial, int blocks, int H,
                                                                   float *__restrict__ dgamma, float *__restrict__ dbeta) {
    __shared__ float s[kSlices][33];
    pdl_trigger();
    pdl_wait();  // the partial sums are visible
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (c < 2 * H)
        for (int b = slice; b < blocks; b += kSlices) sum += partial[static_cast<size_t>(b) * 2 * H + c];
    s[slice][lane] = sum;
    __syncthreads();
    if (slice == 0 && c < 2 * H) {
        for (int k = 1; k < kSlices; ++k) sum += s[k][lane];
        (c < H ? dgamma : dbeta - H)[c] = sum;
    }
}

// Blocks of the gradient and threads of one, one block an SM (as the RMS norm's gradient, rms_norm.cu).
constexpr int kGradBlocks = 152;
constexpr int kGradThreads = 512;
// Threads an SM that the norm's grid is made for (us, 1024 / 2048, without a residual):
// codes per 128 of 12,288 x 7168 88 / 94.5, of 32,768 x 512 16 / 19; rows only, 4096 x
// 2048 14 / 9.6, 16,384 x 1024 18 / 15.4.  (512: 115, 22, 18 and 29.)  2048 are not
// resident at 64 registers a thread: blocks that wait start as soon as others end.
constexpr int kCodeThreadsPerSm = 1024, kPlainThreadsPerSm = 2048;

struct GradShape {
    int vpt, threads, rows;  // vectors a thread, threads a row, rows a block
};
GradShape grad_shape(int64_t H) {
    const int vecs = static_cast<int>(H / 8);
    int vpt = 2;
    while (vpt < 8 && threads_for(vecs, vpt) > 512) vpt *= 2;
    const int threads = threads_for(vecs, vpt);
    // (the shares of dgamma and dbeta of a block with several rows meet in at most 32 KB)
    return {vpt, threads, std::max(1, std::min(kGradThreads / threads, 8))};
}

template <bool BF16>
cudaError_t launch_norm_type(const LayerNormLaunch &p, int kind, int sms, cudaStream_t stream) {
    const int vecs = p.H / 8;
    const auto go = [&](auto launch, int vpt) {
        const int threads = threads_for(vecs, vpt);
        const int per_sm = kind == kQuantNone ? kPlainThreadsPerSm : kCodeThreadsPerSm;
        return launch(p, kind, threads, std::min(p.rows, sms * std::max(1, per_sm / threads)), stream);
    };
    // A vector a thread where all rows are on the SMs at once (its 64 registers leave an
    // SM 1024 threads), and there are no next rows' values to hold.  Without a residual, us,
    // one vector / two: codes per 128 of 1 x 7168 2.5 / 2.7, 128 x 7168 3.2 / 3.9, 152 x
    // 5376 2.8 / 2.9, 304 x 4096 3.1 / 3.3, 600 x 2048 3.3 / 4.6, 2000 x 512 3.2 / 4.1, rows
    // only, 300 x 4096 3.0 / 3.5; past the limit codes 153 x 5376 4.0 / 4.0, 305 x 4096 3.8 /
    // 4.5, 400 x 4096 5.0 / 5.0, 1024 x 4096 8.5 / 7.6, 12,288 x 7168 125 / 87, rows only, 153
    // x 5376 4.2 / 3.1, 200 x 5376 5.2 / 3.5, 400 x 4096 4.6 / 3.9.
    if (vecs <= 1024 && p.rows <= sms * (1024 / threads_for(vecs, 1))) return go(launch_norm_vpt<BF16, 1>, 1);
    if (vecs <= 2048) return go(launch_norm_vpt<BF16, 2>, 2);
    if (vecs <= 4096) return go(launch_norm_vpt<BF16, 4>, 4);
    return go(launch_norm_vpt<BF16, 8>, 8);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormLaunch &p, bool bf16, int kind, int sms, cudaStream_t stream) {
    return bf16 ? launch_norm_type<true>(p, kind, sms, stream) : launch_norm_type<false>(p, kind, sms, stream);
}

// Up to so many turns of their rows by the blocks of one cluster, whose sums are
// then all of them: one launch, no workspace.  The rule is made for eager calls, which
// are bound by the host there: 19 to 21 us against 24 to 26 at all these sizes.  On the
// GPU, in a graph, the two kernels would be faster but for few wide rows (us, cluster /
// two kernels): 9 x 2048 5.0 / 5.0, 32 x 2048 5.6 / 5.1, 128 x 2048 8.2 / 5.6, 16 x 4096
// 5.7 / 5.5, 61 x 4096 8.5 / 5.8, 16 x 7168 6.6 / 6.8, 32 x 7168 8.3 / 6.9, 256 x 1024 8.8 /
// 6.2; four turns of 8 blocks, 61 x 4096, 9.9.
constexpr int kClusterBlocks = 16, kClusterTurns = 2;
constexpr int64_t kClusterWidth = 8192;  // the sums of a block in 64 KB

bool layer_norm_grad_clustered(int64_t rows, int64_t H) {
    return H <= kClusterWidth && rows <= kClusterBlocks * kClusterTurns * grad_shape(H).rows;
}

int layer_norm_grad_blocks(int64_t rows, int64_t H) {
    // Up to two turns of its rows by one block.
    const int64_t r = grad_shape(H).rows;
    if (rows <= 2 * r) return static_cast<int>(std::min<int64_t>(rows, 1));
    return static_cast<int>(std::min<int64_t>((rows + r - 1) / r, layer_norm_grad_clustered(rows, H) ? kClusterBlocks : kGradBlocks));
}

cudaError_t launch_layer_norm_grad(const LayerNormGradLaunch &p, bool bf16, cudaStream_t stream) {
    const GradShape shape = grad_shape(p.H);
    const int cluster = p.clustered && p.blocks > 1 ? p.blocks : 0;
    if (p.blocks > 0) {
        const dim3 block(shape.threads, shape.rows);
        const size_t smem = shape.rows > 1 || cluster ? static_cast<size_t>(p.H) * 8 : 0;
        const auto go = [&](auto kern) {
            cudaError_t err = cudaSuccess;
            if (smem > 48 * 1024)
                err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kClusterWidth) * 8);
            if (err == cudaSuccess && cluster > 8)
                err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            return err == cudaSuccess ? launch_pdl(kern, p.blocks, block, smem, cluster, stream, p) : err;
        };
        cudaError_t err;
        switch (shape.vpt) {
#define A2AV_GRAD(V, MAXT)                                                                                     \
    err = bf16 ? go(layer_norm_grad_kernel<true, V, MAXT>) : go(layer_norm_grad_kernel<false, V, MAXT>); \
    break
            case 2: A2AV_GRAD(2, 512);
            case 4: A2AV_GRAD(4, 512);
            default: A2AV_GRAD(8, 1024);
#undef A2AV_GRAD
        }
        if (err != cudaSuccess) return err;
    }
    if (!p.dgamma || p.blocks == 1 || cluster) return cudaSuccess;
    return launch_pdl(column_sums_kernel, (2 * p.H + 31) / 32, 32 * kSlices, 0, 0, stream,
                      static_cast<const float *>(p.partial), p.blocks, p.H, p.dgamma, p.dbeta);
}

}  // namespace a2av
