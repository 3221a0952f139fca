// The expert layer for a few tokens: the chosen experts' gated blocks (first
// kernel), and their down projections with the weighted sum (second kernel).
//
// Both are bound by the bytes of the weights, which stream from HBM through
// shared memory into the tensor cores as the 128-row operand of tcgen05.mma
// (M, MN-major as they lie in memory); the few rows are the narrow one (N: 16 to
// 64, K-major, copied from where they are by four warps).  The first kernel's
// tile is 64 columns of Wg and the same of Wu; the second's 128 columns of Wd.
// A contraction is cut over the CTAs of a cluster, whose sums are joined in
// order through distributed shared memory: the same result every time.
//
//   first:  a job is (unit, 64 columns); its contraction is H.
//   second: a job is 128 columns of y; its contraction is that of every unit,
//           one behind the other, N each.  A unit's product starts its TMEM
//           accumulator afresh, and is added with the tokens' weights to sums
//           [T][128] in shared memory: what an expert computes reaches its own
//           tokens only.  h comes as two summands of the element type, each
//           multiplied into the same accumulator.
//
// Half of an SM's shared memory at most, so that the second kernel's CTAs stand
// beside the first's while those finish: their weights do not depend on h, and
// are in their stages when the first kernel ends.
// Per CTA: warp 0 loads the weights, warp 1 issues the MMAs, warps 2-5 are the
// epilogue, warps 6-9 copy the rows.  Every wait is bounded.
#include <algorithm>
#include <cmath>

#include "activation.cuh"
#include "moe.h"
#include "moe_plan.cuh"
#include "pair.cuh"
#include "pdl.cuh"
#include "per_device.h"
#include "two_parts.cuh"

namespace a2av {

namespace {

constexpr int kThreads = 10 * 32;
constexpr int kMmaWarp = 1;
constexpr int kEpiWarp0 = 2;
constexpr int kCopyWarp0 = 6;
constexpr int kCopyWarps = 4;
constexpr int kMaxStages = 6;
constexpr int kBK = 64;                       // contraction elements a stage
constexpr uint32_t kAtom = kBK * 128;         // 64 k-rows x 64 columns of weights
constexpr uint32_t kWBytes = 2 * kAtom;
constexpr size_t kSmem = 115712;              // half of an SM's 228 KB, less 1 KB a CTA
static_assert(kThreads >= kMoeExperts, "a thread an expert in the plan");

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t tfull[2], tempty[2];
    uint64_t ready;   // every CTA of the cluster has its part of the sums in shared memory
    uint64_t free;    // every CTA of the cluster has read this CTA's part
    uint32_t tmem_base;
    int32_t abort;
    MoePlan plan;
};
constexpr size_t kControlBytes = (sizeof(Control) + 1023) / 1024 * 1024;

// A stage's rows: R of 64 elements, twice where they come as two summands.
template <bool DOWN, int R>
struct Shape {
    static constexpr int kParts = DOWN ? 2 : 1;
    static constexpr uint32_t kXAtom = R * 128;
    static constexpr uint32_t kStage = kWBytes + kParts * kXAtom;
    static constexpr uint32_t kTmemCols = 2 * R < 32 ? 32 : 2 * R;
    // Rows of the part: the unit's, or the tokens'.
    static int stages(int T) {
        const size_t part = static_cast<size_t>(DOWN ? T : R) * 512;
        return static_cast<int>(std::min<size_t>(kMaxStages, (kSmem - 1024 - kControlBytes - part) / kStage));
    }
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// 16 bytes to shared memory, the first `bytes` of them from src and zeros behind.
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Steps (K blocks) of a job, and the part of them that this CTA takes.
struct Span {
    int begin, end;
};
__device__ __forceinline__ Span span_of(int steps, int rank, int split) {
    return {static_cast<int>(static_cast<int64_t>(steps) * rank / split),
            static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / split)};
}

template <bool BF16, bool DOWN, int ACT, int R>
__global__ void __launch_bounds__(kThreads, 2) moe_rows_kernel(const __grid_constant__ MoeRowsLaunch p) {
    using S = Shape<DOWN, R>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const int stages = p.stages, T = p.choice.T, topk = p.choice.K;
    Control &C = *reinterpret_cast<Control *>(base_ptr + stages * S::kStage);
    float *part = reinterpret_cast<float *>(base_ptr + stages * S::kStage + kControlBytes);  // [R or T][128]
    MoePlan &plan = C.plan;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int split = p.split;  // CTAs of a cluster
    const int rank = static_cast<int>(pair::cluster_rank());
    const int cluster = blockIdx.x / split, clusters = gridDim.x / split;
    const int K = DOWN ? p.N : p.H, cols = DOWN ? p.H : p.N;     // of one product
    constexpr int kJobCols = DOWN ? 128 : 64;
    const int kblocks = (K + kBK - 1) / kBK, strips = (cols + kJobCols - 1) / kJobCols;

    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&C.tmem_base), S::kTmemCols);
        tmem_relinquish();
    } else if (warp == kEpiWarp0) {
        if (lane == 0) {
            for (int s = 0; s < stages; ++s) {
                mbar_init(smem_u32(&C.full[s]), 1 + kCopyWarps);
                mbar_init(smem_u32(&C.empty[s]), 1);
            }
            for (int a = 0; a < 2; ++a) {
                mbar_init(smem_u32(&C.tfull[a]), 1);
                mbar_init(smem_u32(&C.tempty[a]), 4);
            }
            mbar_init(smem_u32(&C.ready), 4 * split);
            mbar_init(smem_u32(&C.free), 4 * split);
            C.abort = 0;
            fence_barrier_init();
        }
    } else if (warp == kEpiWarp0 + 1 && lane == 0) {
        prefetch_tensormap(&p.tmA[0]);
        if (!DOWN) prefetch_tensormap(&p.tmA[1]);
    }
    // The logits are there: the first kernel waits for the router's, and lets the
    // second one start only behind that.
    if (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    moe_plan(p.choice, plan, R, !DOWN && blockIdx.x == 0);
    if (DOWN)
        for (int i = threadIdx.x; i < T * 32; i += kThreads) reinterpret_cast<float4 *>(part)[i] = make_float4(0, 0, 0, 0);
    tc_fence_before_sync();
    pair::sync_all();
    tc_fence_after_sync();

    const int units = plan.units;
    const int jobs = DOWN ? strips : units * strips;
    const Span span = span_of(DOWN ? units * kblocks : kblocks, rank, split);  // the same of every job
    const uint32_t full0 = smem_u32(&C.full[0]), empty0 = smem_u32(&C.empty[0]);
    const uint32_t ready = smem_u32(&C.ready), freed = smem_u32(&C.free);
    const auto unit_of = [&](int job, int step) { return DOWN ? step / kblocks : job / strips; };
    const auto block_of = [&](int step) { return DOWN ? step % kblocks : step; };
    const auto col_of = [&](int job) { return (DOWN ? job : job % strips) * kJobCols; };

    if (warp == 0) {
        // ================================================== producer (weights)
        if (lane == 0) {
            int it = 0;
            bool ok = true, waited = !DOWN;
            for (int job = cluster; job < jobs && ok; job += clusters) {
                const int col = col_of(job);
                for (int step = span.begin; step < span.end; ++step, ++it) {
                    const int s = it % stages;
                    if (!waited && it >= stages) {  // (the time that a wait may take starts behind the kernel before)
                        pdl_wait();
                        waited = true;
                    }
                    if (it >= stages && !pair::wait_phase(&C.abort, empty0 + 8 * s, ((it / stages) & 1) ^ 1, p.status,
                                                          p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = base + s * S::kStage, bar = full0 + 8 * s;
                    const int expert = plan.unit[unit_of(job, step)].expert, k = block_of(step) * kBK;
                    mbar_arrive_expect_tx(bar, kWBytes);
                    tma_load_3d(st, &p.tmA[0], bar, col, k, expert);
                    if (DOWN) tma_load_3d(st + kAtom, &p.tmA[0], bar, col + 64, k, expert);
                    else tma_load_3d(st + kAtom, &p.tmA[1], bar, col, k, expert);
                }
            }
            if (!waited) pdl_wait();
            if (DOWN) pdl_trigger();
            // The stages that were filled have been read.
            for (int i = max(it - stages, 0); i < it && ok; ++i)
                ok = pair::wait_phase(&C.abort, empty0 + 8 * (i % stages), (i / stages) & 1, p.status, p.wait_limit_ns);
            if (!ok) pair::let_settle();
        }
    } else if (warp >= kCopyWarp0) {
        // ================================================== producer (rows)
        // A thread copies the same 16-byte piece of a row's 128 bytes of every 16th
        // row.  The copies are generic-proxy writes, so a stage is handed to the MMA
        // by this thread's fence once they have landed: a stage later, or as soon as
        // there is no stage to fill.
        if (DOWN) pdl_wait();  // h is there
        const int ct = threadIdx.x - kCopyWarp0 * 32, piece = ct % 8, r0 = ct / 8;
        const uint32_t to = r0 * 128 + ((piece ^ (r0 & 7)) << 4);
        const uint16_t *from = static_cast<const uint16_t *>(DOWN ? p.h : p.x);
        const size_t low = static_cast<size_t>(T) * topk * p.N;  // from a first summand to the second
        int it = 0, given = 0;
        bool ok = true;
        const auto hand_over = [&](int until) {
            fence_proxy_async_smem();
            __syncwarp();
            for (; given < until; ++given)
                if (lane == 0) mbar_arrive(full0 + 8 * (given % stages));
        };
        const uint16_t *src[R / 16];
        int unit = -1;
        for (int job = cluster; job < jobs && ok; job += clusters) {
            for (int step = span.begin; step < span.end; ++step, ++it) {
                const int u = unit_of(job, step);
                if (u != unit) {
                    unit = u;
                    const MoeUnit w = plan.unit[u];
#pragma unroll
                    for (int i = 0; i < R / 16; ++i) {
                        const int r = r0 + 16 * i;
                        src[i] = nullptr;  // no such row: zeros
                        if (r < w.rows) {
                            const int pair = plan.pairs[w.first + r];
                            src[i] = from + static_cast<size_t>(DOWN ? pair : pair / topk) * K + piece * 8;
                        }
                    }
                }
                const int s = it % stages;
                const uint32_t par = ((it / stages) & 1) ^ 1;
                // No stage to fill yet: hand over what has been copied rather than wait for more.
                if (given < it && !__all_sync(0xffffffffu, pair::try_wait_cluster(empty0 + 8 * s, par))) {
                    cp_async_wait<0>();
                    hand_over(it);
                }
                if (!pair::wait_phase_warp(&C.abort, empty0 + 8 * s, par, p.status, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t x_st = base + s * S::kStage + kWBytes + to;
                const int k = block_of(step) * kBK;
                const bool in_k = k + piece * 8 < K;
#pragma unroll
                for (int q = 0; q < S::kParts; ++q) {
#pragma unroll
                    for (int i = 0; i < R / 16; ++i) {
                        const bool live = in_k && src[i] != nullptr;
                        cp_async_16_or_zero(x_st + q * S::kXAtom + i * 2048, live ? src[i] + k + q * low : from,
                                            live ? 16 : 0);
                    }
                }
                cp_async_commit();
                if (it - given >= 1) {
                    cp_async_wait<1>();
                    hand_over(it);
                }
            }
        }
        cp_async_wait<0>();
        if (ok) hand_over(it);
    } else if (warp == kMmaWarp) {
        // =========================================================== MMA issuer
        if (lane == 0) {
            if (DOWN) pdl_wait();
            // A: the weights, MN-major (atoms of 64 columns kAtom apart, 8-row K groups 1024 B apart, a K step of 16
            // rows 2 KB).  B: the rows, K-major (8-row groups 1024 B apart, a K step of 16 elements 32 B).
            constexpr uint32_t idesc = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | (1u << 15) |
                                       (static_cast<uint32_t>(R >> 3) << 17) | ((128u >> 4) << 24);
            const uint64_t a_desc0 = smem_desc(base, kAtom, 1024, kSwizzle128B);
            const uint64_t b_desc0 = smem_desc(base + kWBytes, 16, 1024, kSwizzle128B);
            int it = 0, seg = 0;  // stages, accumulators
            bool ok = true;
            for (int job = cluster; job < jobs && ok; job += clusters) {
                for (int step = span.begin; step < span.end; ++step, ++it) {
                    const bool first = step == span.begin || (DOWN && block_of(step) == 0);
                    const bool last = step == span.end - 1 || (DOWN && block_of(step) == kblocks - 1);
                    const int s = it % stages, acc = seg & 1;
                    if ((first && !pair::wait_phase(&C.abort, smem_u32(&C.tempty[acc]), ((seg >> 1) & 1) ^ 1, p.status,
                                                    p.wait_limit_ns)) ||
                        !pair::wait_phase(&C.abort, full0 + 8 * s, (it / stages) & 1, p.status, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t off = (s * S::kStage) >> 4;
                    const int ksteps = (min(kBK, K - block_of(step) * kBK) + 15) / 16;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        if (kk < ksteps) {
#pragma unroll
                            for (int q = 0; q < S::kParts; ++q)
                                mma_f16(C.tmem_base + acc * R, a_desc0 + off + 128 * kk,
                                        b_desc0 + off + ((q * S::kXAtom + kk * 32) >> 4), idesc, !first || kk > 0 || q > 0);
                        }
                    }
                    mma_commit(empty0 + 8 * s);
                    if (last) {
                        mma_commit(smem_u32(&C.tfull[acc]));
                        ++seg;
                    }
                }
            }
        }
    } else {
        // =========================================================== epilogue
        if (DOWN) pdl_wait();
        const int q = warp & 3;  // TMEM lane quarter this warp may read
        const int tid = threadIdx.x - kEpiWarp0 * 32;
        const int own = kJobCols / split;  // columns this CTA finishes
        int jl = 0, seg = 0;
        bool ok = true;
        const auto wait = [&](uint32_t bar, int parity) {
            ok = ok && pair::wait_phase_warp(&C.abort, bar, static_cast<uint32_t>(parity), p.status, p.wait_limit_ns);
            return ok;
        };
        for (int job = cluster; job < jobs && ok; job += clusters, ++jl) {
            // This CTA's part has been read (before it is written again).
            if (!wait(freed, (jl & 1) ^ 1)) break;
            float *const column = part + q * 32 + lane;
            if (DOWN && jl > 0)
                for (int t = 0; t < T; ++t) column[t * 128] = 0.0f;
            if (!DOWN && span.begin == span.end)
                for (int r = 0; r < R; ++r) column[r * 128] = 0.0f;
            // Accumulators of this part: one, or one a unit that it touches.
            for (int step = span.begin; step < span.end; ++seg) {
                const MoeUnit w = plan.unit[unit_of(job, step)];
                if (!wait(smem_u32(&C.tfull[seg & 1]), (seg >> 1) & 1)) break;
                tc_fence_after_sync();
                const uint32_t t_base = C.tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (seg & 1) * R;
#pragma unroll
                for (int c = 0; c < R; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(t_base + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float v = __uint_as_float(r[i]);
                        if (!DOWN) {
                            column[(c + i) * 128] = v;
                        } else if (c + i < w.rows) {
                            const int pair = plan.pairs[w.first + c + i];
                            float *to = column + pair / topk * 128;
                            *to = fmaf(plan.weight[pair], v, *to);
                        }
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&C.tempty[seg & 1]));
                step = DOWN ? min(span.end, (step / kblocks + 1) * kblocks) : span.end;
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0)
                for (int c = 0; c < split; ++c) pair::arrive_cluster(pair::map_to_rank(ready, c));
            if (!wait(ready, jl & 1)) break;
            // This CTA's columns of every row: the parts added in order.
            const int col0 = col_of(job);
            const MoeUnit w = plan.unit[unit_of(job, 0)];
            const int live = DOWN ? T : w.rows;
            for (int i = tid; i < live * own / 4; i += 4 * 32) {
                const int r = i / (own / 4), c = rank * own + i % (own / 4) * 4;
                if (col0 + c >= cols) continue;  // (a multiple of 8: all four columns or none)
                const uint32_t at = smem_u32(part + r * 128 + c);
                float4 g = ld_cluster_f32x4(pair::map_to_rank(at, 0)), u = make_float4(0, 0, 0, 0);
                if (!DOWN) u = ld_cluster_f32x4(pair::map_to_rank(at, 0) + 256);
                for (int k = 1; k < split; ++k) {
                    const uint32_t a = pair::map_to_rank(at, k);
                    const float4 b = ld_cluster_f32x4(a);
                    g = make_float4(g.x + b.x, g.y + b.y, g.z + b.z, g.w + b.w);
                    if (!DOWN) {
                        const float4 d = ld_cluster_f32x4(a + 256);
                        u = make_float4(u.x + d.x, u.y + d.y, u.z + d.z, u.w + d.w);
                    }
                }
                if constexpr (DOWN) {
                    const size_t o = static_cast<size_t>(r) * p.H + col0 + c;
                    f32x2 lo = pair_of(g.x, g.y), hi = pair_of(g.z, g.w);
                    if (p.residual) {
                        const uint2 res = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.residual) + o);
                        lo = add2(lo, unpack2<BF16>(res.x));
                        hi = add2(hi, unpack2<BF16>(res.y));
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + o) = make_uint2(pack2<BF16>(lo), pack2<BF16>(hi));
                } else {
                    float v[4];
                    a2av::split(mul2(act_value<ACT>(pair_of(g.x, g.y)), pair_of(u.x, u.y)), v[0], v[1]);
                    a2av::split(mul2(act_value<ACT>(pair_of(g.z, g.w)), pair_of(u.z, u.w)), v[2], v[3]);
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) two_parts<BF16>(v[k], h[k], l[k]);
                    uint16_t *to = static_cast<uint16_t *>(p.h) +
                                   static_cast<size_t>(plan.pairs[w.first + r]) * p.N + col0 + c;
                    *reinterpret_cast<uint2 *>(to) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                    *reinterpret_cast<uint2 *>(to + static_cast<size_t>(T) * topk * p.N) =
                        make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
                }
            }
            __syncwarp();
            if (lane == 0)
                for (int c = 0; c < split; ++c) pair::arrive_reads_done(pair::map_to_rank(freed, c));
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    pair::sync_all();  // no CTA leaves while another may read its part
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(C.tmem_base, S::kTmemCols);
    }
}

// What a job costs beside its K blocks, in K blocks.
constexpr double kJobCost = 6.0;

// Clusters of 1, 2, 4 and 8 CTAs resident at once.
struct Resident {
    int clusters[4];
};
template <bool DOWN, int R>
const Resident *resident_clusters() {
    static PerDevice<Resident> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
    return cache.get(dev, [](Resident &r) {
        for (int i = 0; i < 4; ++i)
            r.clusters[i] = max_clusters(moe_rows_kernel<true, DOWN, A2AV_ACT_SILU, R>, kThreads, kSmem, 1 << i);
        return r.clusters[0] > 0;
    });
}

template <bool BF16, bool DOWN, int ACT, int R>
cudaError_t launch_rows(MoeRowsLaunch &p, cudaStream_t stream) {
    auto kern = moe_rows_kernel<BF16, DOWN, ACT, R>;
    const cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    const Resident *of_device = resident_clusters<DOWN, R>();
    if (!of_device) return cudaErrorUnknown;
    const MoeChoice &c = p.choice;
    p.stages = Shape<DOWN, R>::stages(c.T);
    // The split of the contraction that takes the least time, counted in K blocks a
    // CTA streams plus what a job costs beside them, for the experts that choices
    // at random would reach.
    const double reached = c.E * (1.0 - std::pow(1.0 - static_cast<double>(c.K) / c.E, static_cast<double>(c.T)));
    const int strips = DOWN ? (p.H + 127) / 128 : (p.N + 63) / 64;
    const double jobs = DOWN ? strips : std::ceil(reached - 0.5) * strips;
    const double steps = DOWN ? std::ceil(reached - 0.5) * ((p.N + kBK - 1) / kBK) : (p.H + kBK - 1) / kBK;
    double best = 0.0;
    for (int i = 0; i < 4; ++i) {
        const int resident = of_device->clusters[i];
        if (resident <= 0) continue;
        const double cost = std::ceil(jobs / resident) * (std::ceil(steps / (1 << i)) + kJobCost);
        if (p.split == 0 || cost < best) {
            best = cost;
            p.split = 1 << i;
            p.grid = resident << i;
        }
    }
    const int64_t most_jobs = DOWN ? strips : static_cast<int64_t>(c.T) * c.K * strips;
    p.grid = static_cast<int>(std::min<int64_t>(p.grid, most_jobs * p.split));
    return launch_pdl(kern, dim3(p.grid), dim3(kThreads), kSmem, p.split, stream, p);
}

// Rows of a unit: what the fullest expert is expected to have, so that one pass
// over its weights is usual.
template <bool BF16, bool DOWN, int ACT>
cudaError_t launch_unit(MoeRowsLaunch &p, cudaStream_t stream) {
    const double mean = static_cast<double>(p.choice.T) * p.choice.K / p.choice.E;
    const double most = std::min<double>(p.choice.T, mean + 3.0 * std::sqrt(mean) + 1.0);
    if (most <= 16) return launch_rows<BF16, DOWN, ACT, 16>(p, stream);
    if (most <= 32) return launch_rows<BF16, DOWN, ACT, 32>(p, stream);
    return launch_rows<BF16, DOWN, ACT, 64>(p, stream);
}

}  // namespace

cudaError_t launch_moe_gated(MoeRowsLaunch p, bool bf16, int act, cudaStream_t stream) {
    p.split = 0;
    if (bf16)
        return act == A2AV_ACT_SILU ? launch_unit<true, false, A2AV_ACT_SILU>(p, stream)
                                    : launch_unit<true, false, A2AV_ACT_GELU_TANH>(p, stream);
    return act == A2AV_ACT_SILU ? launch_unit<false, false, A2AV_ACT_SILU>(p, stream)
                                : launch_unit<false, false, A2AV_ACT_GELU_TANH>(p, stream);
}

cudaError_t launch_moe_down(MoeRowsLaunch p, bool bf16, cudaStream_t stream) {
    p.split = 0;
    return bf16 ? launch_unit<true, true, A2AV_ACT_SILU>(p, stream) : launch_unit<false, true, A2AV_ACT_SILU>(p, stream);
}

}  // namespace a2av
