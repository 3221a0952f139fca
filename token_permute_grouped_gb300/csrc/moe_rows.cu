// The expert layer for a few tokens: the chosen experts' gated blocks (first
// kernel), and their down projections with the weighted sum (second kernel).
//
// Both are bound by the bytes of the weights, which stream from HBM through
// shared memory into the tensor cores as the 128-row operand of tcgen05.mma
// (M, MN-major as they lie in memory); the few rows are the narrow one (N: 16 to
// 64, K-major).  The first kernel's tile is 64 columns of Wg and the same of Wu;
// the second's 128 columns of Wd.  A contraction is cut over the CTAs of a
// cluster, whose sums are joined in order through distributed shared memory: the
// same result every time.
//
//   first:  a job is (expert, 64 columns); its contraction is H.  All tokens are
//           multiplied, which costs nothing beside the weights and needs no
//           gathering; the rows of those that chose the expert are kept, and
//           stored expert after expert.
//   second: a job is 128 columns of y; its contraction is that of every unit (up
//           to R rows of an expert, which lie together), one behind the other, N
//           each.  A unit's product starts its TMEM accumulator afresh, and is
//           added with the tokens' weights to sums [T][128] in shared memory:
//           what an expert computes reaches its own tokens only.  h comes as two
//           summands of the element type, each multiplied into the same
//           accumulator.
//
// Half of an SM's shared memory at most, so that the second kernel's CTAs stand
// beside the first's while those finish: their weights do not depend on h, and
// are in their stages when the first kernel ends.
// Per CTA: warp 0 loads, warp 1 issues the MMAs, warps 2-5 are the epilogue (all
// eight make the plan).  Every wait is bounded.
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

constexpr int kThreads = 8 * 32;
constexpr int kMmaWarp = 1;
constexpr int kEpiWarp0 = 2;
constexpr int kEpiWarps = 4;
constexpr int kGroup = 16;                    // rows that the first kernel finishes at a time
constexpr int kMaxStages = 6;
constexpr int kBK = 64;                       // contraction elements a stage
constexpr uint32_t kAtom = kBK * 128;         // 64 k-rows x 64 columns of weights
constexpr uint32_t kWBytes = 2 * kAtom;
constexpr size_t kSmem = 114688;              // two CTAs an SM
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
    // Rows of the part: a group's, or the tokens'.
    static int stages(int T) {
        const size_t part = static_cast<size_t>(DOWN ? T : kGroup) * 512;
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// One lane of the (whole) warp.
__device__ __forceinline__ bool elect() {
    uint32_t is;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(is));
    return is != 0;
}

// One column.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
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
    float *part = reinterpret_cast<float *>(base_ptr + stages * S::kStage + kControlBytes);  // [kGroup or T][128]
    MoePlan &plan = C.plan;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
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
                mbar_init(smem_u32(&C.full[s]), 1);
                mbar_init(smem_u32(&C.empty[s]), 1);
            }
            for (int a = 0; a < 2; ++a) {
                mbar_init(smem_u32(&C.tfull[a]), 1);
                mbar_init(smem_u32(&C.tempty[a]), kEpiWarps);
            }
            mbar_init(smem_u32(&C.ready), kEpiWarps * split);
            mbar_init(smem_u32(&C.free), kEpiWarps * split);
            C.abort = 0;
            fence_barrier_init();
        }
    } else if (warp == kEpiWarp0 + 1 && lane == 0) {
        prefetch_tensormap(&p.tmA[0]);
        prefetch_tensormap(&p.tmX);
        if (!DOWN) prefetch_tensormap(&p.tmA[1]);
    }
    // The logits are there: the first kernel waits for the router's, and lets the
    // second one start only behind that.
    if (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    moe_plan(p.choice, plan, DOWN ? R : kMoeTokens, !DOWN && blockIdx.x == 0);
    if (DOWN)
        for (int i = threadIdx.x; i < T * 32; i += kThreads) reinterpret_cast<float4 *>(part)[i] = make_float4(0, 0, 0, 0);
    tc_fence_before_sync();
    pair::sync_all();
    tc_fence_after_sync();

    const int units = __shfl_sync(0xffffffffu, plan.units, 0);
    const int jobs = DOWN ? strips : units * strips;
    const Span span = span_of(DOWN ? units * kblocks : kblocks, rank, split);  // the same of every job
    const uint32_t full0 = smem_u32(&C.full[0]), empty0 = smem_u32(&C.empty[0]);
    const uint32_t ready = smem_u32(&C.ready), freed = smem_u32(&C.free);
    const auto unit_of = [&](int job, int step) { return DOWN ? step / kblocks : job / strips; };
    const auto col_of = [&](int job) { return (DOWN ? job : job % strips) * kJobCols; };
    // A ring's place: stage and how often it has been gone round.
    struct Place {
        int s = 0, turn = 0;
        __device__ __forceinline__ void next(int n) {
            if (++s == n) s = 0, ++turn;
        }
    };

    if (warp == 0) {
        // =========================================================== producer
        // (The whole warp goes along and one lane issues, which leaves the operands in
        // uniform registers: an MMA or a load that a branch on the lane issues costs
        // two to four times the slots.)
        const bool leader = elect();
        constexpr uint32_t kXBytes = S::kParts * S::kXAtom;
        const auto weights = [&](const Place &at, int job, int unit, int block) {
            const uint32_t st = base + at.s * S::kStage, bar = full0 + 8 * at.s;
            const int expert = plan.unit[unit].expert, col = col_of(job), k = block * kBK;
            if (leader) {
                mbar_arrive_expect_tx(bar, kWBytes + kXBytes);
                tma_load_3d(st, &p.tmA[0], bar, col, k, expert);
                if (DOWN) tma_load_3d(st + kAtom, &p.tmA[0], bar, col + 64, k, expert);
                else tma_load_3d(st + kAtom, &p.tmA[1], bar, col, k, expert);
            }
        };
        const auto rows = [&](const Place &at, int unit, int block) {
            const uint32_t st = base + at.s * S::kStage, bar = full0 + 8 * at.s;
            const int first = DOWN ? plan.unit[unit].first : 0;
            if (leader) tma_load_3d(st + kWBytes, &p.tmX, bar, block * kBK, first, 0);
        };
        bool ok = true;
        // The second kernel's first stages: their weights before the first kernel's
        // end, the rows behind it.  (The time that a wait may take starts there.)
        const int first_unit = DOWN ? span.begin / kblocks : 0, first_block = DOWN ? span.begin % kblocks : span.begin;
        const int ahead = DOWN && cluster < jobs ? min(stages, span.end - span.begin) : 0;
        if (DOWN) {
            for (int pass = 0; pass < 2; ++pass) {
                if (pass == 1) pdl_wait();
                Place at;
                int unit = first_unit, block = first_block;
                for (int i = 0; i < ahead; ++i) {
                    if (pass == 0) weights(at, cluster, unit, block);
                    else rows(at, unit, block);
                    at.next(stages);
                    if (++block == kblocks) block = 0, ++unit;
                }
            }
        }
        Place at;
        int filled = 0;
        for (int job = cluster; job < jobs && ok; job += clusters) {
            int unit = DOWN ? first_unit : job / strips, block = first_block;
            for (int step = span.begin; step < span.end; ++step) {
                if (filled >= ahead) {
                    if (at.turn > 0 && !pair::wait_phase_warp(&C.abort, empty0 + 8 * at.s, (at.turn & 1) ^ 1, p.status,
                                                              p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    weights(at, job, unit, block);
                    rows(at, unit, block);
                }
                ++filled;
                at.next(stages);
                if (++block == kblocks) block = 0, ++unit;
            }
        }
        if (DOWN) pdl_trigger();
        // The stages that were filled have been read.
        for (int i = 0; i < stages && ok; ++i) {
            const int turns = at.s > i ? at.turn + 1 : at.turn;  // fills of stage i
            if (turns > 0)
                ok = pair::wait_phase_warp(&C.abort, empty0 + 8 * i, (turns - 1) & 1, p.status, p.wait_limit_ns);
        }
        if (!ok) pair::let_settle();
    } else if (warp == kMmaWarp) {
        // =========================================================== MMA issuer
        if (DOWN) pdl_wait();
        const bool leader = elect();
        // A: the weights, MN-major (atoms of 64 columns kAtom apart, 8-row K groups 1024 B apart, a K step of 16
        // rows 2 KB).  B: the rows, K-major (8-row groups 1024 B apart, a K step of 16 elements 32 B).
        constexpr uint32_t idesc = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | (1u << 15) |
                                   (static_cast<uint32_t>(R >> 3) << 17) | ((128u >> 4) << 24);
        const uint64_t a_desc0 = smem_desc(base, kAtom, 1024, kSwizzle128B);
        const uint64_t b_desc0 = smem_desc(base + kWBytes, 16, 1024, kSwizzle128B);
        const uint32_t tmem = __shfl_sync(0xffffffffu, C.tmem_base, 0);
        Place at;
        int seg = 0;  // accumulators
        bool ok = true;
        for (int job = cluster; job < jobs && ok; job += clusters) {
            int block = DOWN ? span.begin % kblocks : span.begin;
            for (int step = span.begin; step < span.end; ++step) {
                const bool first = step == span.begin || (DOWN && block == 0);
                const bool last = step == span.end - 1 || (DOWN && block == kblocks - 1);
                const int acc = seg & 1;
                if ((first && !pair::wait_phase_warp(&C.abort, smem_u32(&C.tempty[acc]), ((seg >> 1) & 1) ^ 1, p.status,
                                                     p.wait_limit_ns)) ||
                    !pair::wait_phase_warp(&C.abort, full0 + 8 * at.s, at.turn & 1, p.status, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint64_t off = static_cast<uint32_t>(at.s * S::kStage) >> 4;
                const int ksteps = (min(kBK, K - block * kBK) + 15) / 16;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        if (kk < ksteps) {
#pragma unroll
                            for (int q = 0; q < S::kParts; ++q)
                                mma_f16(tmem + acc * R, a_desc0 + off + 128 * kk,
                                        b_desc0 + off + ((q * S::kXAtom + kk * 32) >> 4), idesc, !first || kk > 0 || q > 0);
                        }
                    }
                    mma_commit(empty0 + 8 * at.s);
                    if (last) mma_commit(smem_u32(&C.tfull[acc]));
                }
                __syncwarp();
                if (last) ++seg;
                at.next(stages);
                if (++block == kblocks) block = 0;
            }
        }
    } else if (warp < kEpiWarp0 + kEpiWarps) {
        // =========================================================== epilogue
        if (DOWN) pdl_wait();
        const int q = warp & 3;  // TMEM lane quarter this warp may read
        const int tid = threadIdx.x - kEpiWarp0 * 32;
        const int own = kJobCols / split;  // columns this CTA finishes
        const uint32_t t_base = C.tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        float *const column = part + q * 32 + lane;
        int round = 0, seg = 0;  // exchanges over the cluster, accumulators
        bool ok = true;
        const auto wait = [&](uint32_t bar, int parity) {
            ok = ok && pair::wait_phase_warp(&C.abort, bar, static_cast<uint32_t>(parity), p.status, p.wait_limit_ns);
            return ok;
        };
        const auto released = [&]() {  // an accumulator has been read
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&C.tempty[seg & 1]));
            ++seg;
        };
        // Every CTA's part is there.
        const auto exchanged = [&]() {
            __syncwarp();
            if (lane == 0)
                for (int c = 0; c < split; ++c) pair::arrive_cluster(pair::map_to_rank(ready, c));
            return wait(ready, round & 1);
        };
        const auto parts_read = [&]() {
            __syncwarp();
            if (lane == 0)
                for (int c = 0; c < split; ++c) pair::arrive_reads_done(pair::map_to_rank(freed, c));
            ++round;
        };
        for (int job = cluster; job < jobs && ok; job += clusters) {
            const int col0 = col_of(job);
            if constexpr (!DOWN) {
                const MoeUnit w = plan.unit[unit_of(job, 0)];
                const bool any = span.begin < span.end;
                if (any) {
                    if (!wait(smem_u32(&C.tfull[seg & 1]), (seg >> 1) & 1)) break;
                    tc_fence_after_sync();
                }
                for (int g = 0; g < w.rows; g += kGroup) {
                    const int live = min(kGroup, w.rows - g);
                    uint32_t v[kGroup];
                    if (any) {
#pragma unroll
                        for (int i = 0; i < kGroup; ++i)
                            if (i < live) tmem_ld1(t_base + (seg & 1) * R + plan.pairs[w.first + g + i] / topk, v[i]);
                        tmem_ld_wait();
                    }
                    // This CTA's part has been read (before it is written again).
                    if (!wait(freed, (round & 1) ^ 1)) break;
#pragma unroll
                    for (int i = 0; i < kGroup; ++i)
                        if (i < live) column[i * 128] = any ? __uint_as_float(v[i]) : 0.0f;
                    if (any && g + kGroup >= w.rows) released();
                    if (!exchanged()) break;
                    // This CTA's columns of every row: the parts added in order.
                    for (int i = tid; i < live * own / 4; i += kEpiWarps * 32) {
                        const int r = i / (own / 4), c = rank * own + i % (own / 4) * 4;
                        if (col0 + c >= cols) continue;  // (a multiple of 8: all four columns or none)
                        const uint32_t at = smem_u32(part + r * 128 + c);
                        f32x2 s[4] = {0, 0, 0, 0};
                        for (int k = 0; k < split; ++k) {
                            const uint32_t a = pair::map_to_rank(at, k);
                            const float4 b = ld_cluster_f32x4(a), d = ld_cluster_f32x4(a + 256);
                            s[0] = add2(s[0], pair_of(b.x, b.y));
                            s[1] = add2(s[1], pair_of(b.z, b.w));
                            s[2] = add2(s[2], pair_of(d.x, d.y));
                            s[3] = add2(s[3], pair_of(d.z, d.w));
                        }
                        float f[4];
                        a2av::split(mul2(act_value<ACT>(s[0]), s[2]), f[0], f[1]);
                        a2av::split(mul2(act_value<ACT>(s[1]), s[3]), f[2], f[3]);
                        uint32_t h[4], l[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) two_parts<BF16>(f[k], h[k], l[k]);
                        uint16_t *to = static_cast<uint16_t *>(p.h) + static_cast<size_t>(w.first + g + r) * p.N + col0 + c;
                        *reinterpret_cast<uint2 *>(to) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                        *reinterpret_cast<uint2 *>(to + static_cast<size_t>(T) * topk * p.N) =
                            make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
                    }
                    parts_read();
                }
            } else {
                if (!wait(freed, (round & 1) ^ 1)) break;
                if (round > 0)
                    for (int t = 0; t < T; ++t) column[t * 128] = 0.0f;
                for (int step = span.begin; step < span.end; step = min(span.end, (step / kblocks + 1) * kblocks)) {
                    const MoeUnit w = plan.unit[unit_of(job, step)];
                    if (!wait(smem_u32(&C.tfull[seg & 1]), (seg >> 1) & 1)) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int c = 0; c < R; c += 16) {
                        if (c < w.rows) {
                            uint32_t r[16];
                            tmem_ld16(t_base + (seg & 1) * R + c, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                if (c + i < w.rows) {
                                    const int pair = plan.pairs[w.first + c + i];
                                    float *to = column + pair / topk * 128;
                                    *to = fmaf(plan.weight[pair], __uint_as_float(r[i]), *to);
                                }
                            }
                        }
                    }
                    released();
                }
                if (!ok || !exchanged()) break;
                for (int i = tid; i < T * own / 4; i += kEpiWarps * 32) {
                    const int r = i / (own / 4), c = rank * own + i % (own / 4) * 4;
                    if (col0 + c >= cols) continue;
                    const uint32_t at = smem_u32(part + r * 128 + c);
                    f32x2 s[2] = {0, 0};
                    for (int k = 0; k < split; ++k) {
                        const float4 b = ld_cluster_f32x4(pair::map_to_rank(at, k));
                        s[0] = add2(s[0], pair_of(b.x, b.y));
                        s[1] = add2(s[1], pair_of(b.z, b.w));
                    }
                    const size_t o = static_cast<size_t>(r) * p.H + col0 + c;
                    if (p.residual) {
                        const uint2 res = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.residual) + o);
                        s[0] = add2(s[0], unpack2<BF16>(res.x));
                        s[1] = add2(s[1], unpack2<BF16>(res.y));
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + o) =
                        make_uint2(pack2<BF16>(s[0]), pack2<BF16>(s[1]));
                }
                parts_read();
            }
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

// Clusters of 1, 2, 4 and 8 CTAs resident at once: twice what the query answers,
// which takes a kernel with TMEM to have an SM for itself (two CTAs of up to 256
// columns do share one).
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
            r.clusters[i] = 2 * max_clusters(moe_rows_kernel<true, DOWN, A2AV_ACT_SILU, R>, kThreads, kSmem, 1 << i);
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

// Rows multiplied: all tokens, or a unit's: what the fullest expert is expected
// to have, so that one pass over its weights is usual.
template <bool BF16, bool DOWN, int ACT>
cudaError_t launch_unit(MoeRowsLaunch &p, cudaStream_t stream) {
    const int R = moe_unit_rows(p.choice.T, p.choice.E, p.choice.K, DOWN);
    if (R == 16) return launch_rows<BF16, DOWN, ACT, 16>(p, stream);
    if (R == 32) return launch_rows<BF16, DOWN, ACT, 32>(p, stream);
    return launch_rows<BF16, DOWN, ACT, 64>(p, stream);
}

}  // namespace

int moe_unit_rows(int T, int E, int K, bool down) {
    const double mean = static_cast<double>(T) * K / E;
    const double most = down ? std::min<double>(T, mean + 3.0 * std::sqrt(mean) + 1.0) : T;
    return most <= 16 ? 16 : most <= 32 ? 32 : 64;
}

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
