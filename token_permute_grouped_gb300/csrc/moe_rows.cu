// The expert layer for a few tokens: the chosen experts' gated blocks (first
// kernel), and their down projections with the weighted sum (second kernel).
//
// Both are bound by the bytes of the weights, which stream from HBM through
// shared memory into the tensor cores as the 128-row operand of tcgen05.mma
// (M, MN-major as they lie in memory); the few rows are the narrow one (N: 16 to
// 64, K-major).  A tile is 128 columns of a matrix: CTAs beside each other read
// different places, and 256 bytes of a weight's row at a time come at 6.8 TB/s
// from HBM where 128 come at 5.5.
//
//   first:  a job is (expert, 128 columns); its contraction is H, each K block one
//           of Wg and one of Wu, into an accumulator each.  All tokens are
//           multiplied, which costs nothing beside the weights and needs no
//           gathering; the rows of those that chose the expert are kept, and
//           stored expert after expert.
//   second: a job is 128 columns of y; its contraction is that of every unit (up
//           to R rows of an expert, which lie together), one behind the other, N
//           each.  A unit's product starts its TMEM accumulator afresh, and is
//           added with the tokens' weights to sums [T][128] in shared memory:
//           what an expert computes reaches its own tokens only.  h comes as two
//           summands of the element type (value_parts).
//
// How many experts are reached is known on the device only, so the K blocks of
// all jobs, one behind the other, are cut into one equal piece a CTA.  A job that
// several CTAs share has its sums put into the workspace by each; the last of
// them to come adds all in order: the same result every time, whoever it is.  For
// many tokens the second kernel's shares are added by a third one, in the same order.
//
// The second kernel's weights do not depend on h, and fill the stages of a CTA as
// soon as the first kernel's have left its SM.  (Half of an SM's shared memory each,
// so that they stand beside each other from the start, was no faster for one token
// over 32 experts of 2048 x 1024, and 5 to 11% slower for 16 to 32.)
//
// Measured with the router's two kernels (weights from HBM, us; in brackets what the
// weights of all experts would take at a plain copy's 6.68 TB/s): 1 token, 4 of 32
// experts of 2048 x 1024 27; 32 tokens 82 to 87 [60]; 1 token, 6 of 64 of 2048 x 1408 37,
// 32 tokens 178 [166]; 1 token, 2 of 8 of 4096 x 4096 50, 32 tokens 150 [121].
// Per CTA: warps 0, 6 and 7 load, warp 1 issues the MMAs, warps 2-5 are the
// epilogue (all eight make the plan).  Every wait is bounded.
#include <algorithm>
#include <cmath>

#include "activation.cuh"
#include "moe.h"
#include "moe_plan.cuh"
#include "pair.cuh"
#include "pdl.cuh"
#include "two_parts.cuh"

namespace a2av {

namespace {

constexpr int kThreads = 8 * 32;
// Tokens up to which the last CTA of a job of the second kernel adds its shares; above,
// a kernel behind it (us, last CTA / kernel: 1 token, 7 of 49 experts of 384 x 384 19 /
// 24, 4 of 32 of 2048 x 1024 27 / 28; 8 tokens 31.5 / 40, 59 / 61; 16 tokens 45 / 40, 78 /
// 80; 64 tokens 89 / 48, 102 / 91).
constexpr int kAloneTokens = 8;
constexpr int kMmaWarp = 1;
constexpr int kEpiWarp0 = 2;
constexpr int kEpiWarps = 4;
constexpr int kLoadWarp1 = kEpiWarp0 + kEpiWarps;  // loads beside warp 0, and the one behind it
constexpr int kLoadWarps = 3;
constexpr int kGroup = 8;                     // rows that the first kernel finishes at a time
constexpr int kMaxStages = 10;
constexpr int kBK = 64;                       // contraction elements a stage
constexpr uint32_t kAtom = kBK * 128;         // 64 k-rows x 64 columns of weights
constexpr uint32_t kWBytes = 2 * kAtom;
constexpr size_t kSmem = 231424;
static_assert(kThreads >= kMoeExperts, "a thread an expert in the plan");

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t tfull[2], tempty[2];
    uint32_t tmem_base;
    int32_t abort;
    int32_t arrived;  // what this CTA's arrival at a shared job found
    MoePlan plan;
};
constexpr size_t kControlBytes = (sizeof(Control) + 1023) / 1024 * 1024;

// A value of the gated block as two summands of the element type for the second
// product, which has the other factor in that type.  bf16: value = h + l, into one
// accumulator (two_parts.cuh: 2^-15 of the value and less).  fp16: value = 2 h + l / 1024,
// into an accumulator each, which are added as fp32: one scale for both would take
// values below 1e-4 for multiples of fp16's least, 6e-8.  So a value is held to 2^-22 of
// it or 2^-35, from 0 to twice fp16's range, and is infinite beyond.  h is 0 for 0 only:
// an infinite weight makes h's sum infinite or NaN, which is then the product's (l may
// have the other sign).
constexpr float kHigh = 2.0f, kLow = 1.0f / 1024.0f;
template <bool BF16>
__device__ __forceinline__ void value_parts(float v, uint32_t &h, uint32_t &l) {
    if constexpr (BF16) {
        two_parts<true>(v, h, l);
    } else {
        h = __half_as_ushort(__float2half_rn(v / kHigh));
        if ((h & 0x7fffu) == 0 && v != 0.0f) h = v < 0.0f ? 0x8001u : 1u;
        const float high = kHigh * __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
        l = (h & 0x7fffu) < 0x7c00u ? __half_as_ushort(__float2half_rn((v - high) / kLow)) : 0u;
    }
}
__device__ __forceinline__ float sum_of_parts(float h, float l) {
    return fabsf(h) < __uint_as_float(0x7f800000u) ? fmaf(kHigh, h, kLow * l) : h;
}

// A stage's rows: R of 64 elements, twice where they come as two summands.  A K
// block is a stage of each matrix.  The gate's and the up projection's products have an
// accumulator each, and so have fp16's summands.
template <bool BF16, bool DOWN, int R>
struct Shape {
    static constexpr int kMats = DOWN ? 1 : 2;
    static constexpr int kParts = DOWN ? 2 : 1;
    static constexpr bool kApart = DOWN && !BF16;
    static constexpr uint32_t kXAtom = R * 128;
    static constexpr uint32_t kStage = kWBytes + kParts * kXAtom;
    static constexpr uint32_t kAccCols = (kApart ? 2 : kMats) * R;  // of a set of accumulators, of which there are two
    static constexpr uint32_t kTmemCols = 2 * kAccCols;
    static int stages(int T) {
        const size_t part = DOWN ? static_cast<size_t>(T) * 512 : 0;  // the tokens' sums
        return static_cast<int>(std::min<size_t>(kMaxStages, (kSmem - 1024 - kControlBytes - part) / kStage));
    }
};

// One column, and the wait behind which a group of them is used.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_ld1_wait(uint32_t (&r)[kGroup][2]) {
    static_assert(kGroup == 8, "as many registers below");
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0][0]), "+r"(r[0][1]), "+r"(r[1][0]), "+r"(r[1][1]), "+r"(r[2][0]), "+r"(r[2][1]),
                   "+r"(r[3][0]), "+r"(r[3][1]), "+r"(r[4][0]), "+r"(r[4][1]), "+r"(r[5][0]), "+r"(r[5][1]),
                   "+r"(r[6][0]), "+r"(r[6][1]), "+r"(r[7][0]), "+r"(r[7][1])
                 :
                 : "memory");
}

// A K block among all jobs'.
struct Cursor {
    int job, unit, block;
};

// All threads of the epilogue.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory"); }
// The same, and whether all of them say yes: a warp whose wait was given up takes the others along.
__device__ __forceinline__ bool epilogue_all(bool yes) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 2, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(static_cast<uint32_t>(yes)), "n"(kEpiWarps * 32)
        : "memory");
    return all != 0;
}

// CTAs among which the K blocks of all jobs are cut: a CTA has one at least, so
// that a job's shares are those of consecutive CTAs.  The first kernel's shares are
// added by one CTA, about 0.02 us for a row of each, and a K block takes a CTA 0.32
// us: more CTAs a job than make the sum of both least are not used.  (With all, 16
// tokens at each of 4 experts of 3288 x 192: 48 us against 39.)
template <bool DOWN>
__device__ __forceinline__ int moe_ctas(const MoeChoice &c, int grid, int units, int strips, int kblocks) {
    const int64_t total = static_cast<int64_t>(units) * strips * kblocks;
    int ctas = static_cast<int>(min(static_cast<int64_t>(grid), total));
    if (!DOWN) {
        const float rows = static_cast<float>(c.T * c.K) / static_cast<float>(units);  // of a job
        const float shares = fmaxf(1.0f, sqrtf(16.0f * static_cast<float>(kblocks) / rows));
        ctas = static_cast<int>(fminf(static_cast<float>(ctas), ceilf(static_cast<float>(units * strips) * shares)));
    }
    return ctas;
}

template <bool BF16, bool DOWN, int ACT, int R>
__global__ void __launch_bounds__(kThreads, 1) moe_rows_kernel(const __grid_constant__ MoeRowsLaunch p) {
    using S = Shape<BF16, DOWN, R>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const int stages = p.stages, T = p.choice.T, topk = p.choice.K;
    Control &C = *reinterpret_cast<Control *>(base_ptr + stages * S::kStage);
    float *part = reinterpret_cast<float *>(base_ptr + stages * S::kStage + kControlBytes);  // second: [T][128]
    MoePlan &plan = C.plan;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int K = DOWN ? p.N : p.H, cols = DOWN ? p.H : p.N;  // of one product
    constexpr int kJobCols = 128;
    const int kblocks = (K + kBK - 1) / kBK, strips = (cols + kJobCols - 1) / kJobCols;

    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&C.tmem_base), S::kTmemCols);
        tmem_relinquish();
    } else if (warp == kEpiWarp0) {
        if (lane == 0) {
            for (int s = 0; s < stages; ++s) {
                mbar_init(smem_u32(&C.full[s]), kLoadWarps);
                mbar_init(smem_u32(&C.empty[s]), 1);
            }
            for (int a = 0; a < 2; ++a) {
                mbar_init(smem_u32(&C.tfull[a]), 1);
                mbar_init(smem_u32(&C.tempty[a]), kEpiWarps);
            }
            C.abort = 0;
            fence_barrier_init();
        }
    } else if (warp == kEpiWarp0 + 1 && lane == 0) {
        prefetch_tensormap(&p.tmA[0]);
        prefetch_tensormap(&p.tmX);
        if (!DOWN) prefetch_tensormap(&p.tmA[1]);
    }
    // The choice is there: the first kernel waits for it, and lets the second one start
    // only behind that.
    if (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    moe_plan(p.choice, plan, DOWN ? R : kMoeTokens);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();

    const int units = __shfl_sync(0xffffffffu, plan.units, 0);
    // The K blocks of all jobs, and this CTA's.
    const int length = DOWN ? units * kblocks : kblocks;  // of a job
    const int64_t total = static_cast<int64_t>(DOWN ? strips : units * strips) * length;
    const int ctas = moe_ctas<DOWN>(p.choice, gridDim.x, units, strips, kblocks), me = blockIdx.x;
    const auto begin_of = [&](int cta) { return static_cast<int>(total * cta / ctas); };
    const auto owner_of = [&](int step) { return static_cast<int>(((step + 1ll) * ctas - 1) / total); };
    const int begin = me < ctas ? begin_of(me) : 0, end = me < ctas ? begin_of(me + 1) : 0;
    Cursor first;
    first.job = begin / length;
    first.unit = DOWN ? begin % length / kblocks : first.job / strips;
    first.block = begin % kblocks;
    const auto advance = [&](Cursor &c) {
        if (++c.block < kblocks) return;
        c.block = 0;
        if (DOWN) {
            if (++c.unit == units) c.unit = 0, ++c.job;
        } else {
            c.unit = ++c.job / strips;
        }
    };
    const auto col_of = [&](int job) { return (DOWN ? job : job % strips) * kJobCols; };
    const uint32_t full0 = smem_u32(&C.full[0]), empty0 = smem_u32(&C.empty[0]);
    // A ring's place: stage and how often it has been gone round.
    struct Place {
        int s = 0, turn = 0;
        __device__ __forceinline__ void next(int n) {
            if (++s == n) s = 0, ++turn;
        }
    };

    if (DOWN && me == 0 && threadIdx.x == 0) *p.units = units;  // (for the kernel that joins)

    if (warp == 0 || warp >= kLoadWarp1) {
        // =========================================================== producers
        // Three warps issue a load a stage each (a warp takes about 240 clocks for one):
        // the two atoms of weights, and the rows.  A whole warp goes along and one lane
        // issues, which leaves the operands in uniform registers: an MMA that a branch
        // on the lane issues costs two to four times the slots.
        const int what = warp == 0 ? 0 : warp - kLoadWarp1 + 1;
        const bool leader = elect_one();
        const uint32_t bytes = what == 2 ? S::kParts * S::kXAtom : kAtom, to = base + what * kAtom;
        const int shift = what == 1 ? 64 : 0;  // of the columns
        // The second kernel's first stages: their weights before the first kernel's
        // end, the rows behind it.  (The time that a wait may take starts there.)
        const int ahead = DOWN && what != 2 ? min(stages, end - begin) : 0;
        bool ok = true;
        Place at;
        Cursor c = first;
        int col = col_of(c.job) + shift, group = what == 2 ? 0 : plan.unit[c.unit].expert;
        int row = what == 2 && DOWN ? plan.unit[c.unit].first : 0;
        for (int step = begin; step < end && ok; ++step) {
            if (DOWN && step == begin + ahead) pdl_wait();
#pragma unroll
            for (int m = 0; m < S::kMats; ++m) {
                if (at.turn > 0 && !pair::wait_phase_warp(&C.abort, empty0 + 8 * at.s, (at.turn & 1) ^ 1, p.status,
                                                          p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = full0 + 8 * at.s, dst = to + at.s * S::kStage;
                if (leader) {
                    mbar_arrive_expect_tx(bar, bytes);
                    if (what == 2) tma_load_3d(dst, &p.tmX, bar, c.block * kBK, row, 0);
                    else tma_load_3d(dst, &p.tmA[m], bar, col, c.block * kBK, group);
                }
                __syncwarp();
                at.next(stages);
            }
            advance(c);
            if (c.block == 0 && step + 1 < end) {
                if (what != 2) col = col_of(c.job) + shift, group = plan.unit[c.unit].expert;
                else if (DOWN) row = plan.unit[c.unit].first;
            }
        }
        if (DOWN && end - begin <= ahead) pdl_wait();
        if (DOWN && what == 0) pdl_trigger();
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
        const bool leader = elect_one();
        // A: the weights, MN-major (atoms of 64 columns kAtom apart, 8-row K groups 1024 B apart, a K step of 16
        // rows 2 KB).  B: the rows, K-major (8-row groups 1024 B apart, a K step of 16 elements 32 B).
        constexpr uint32_t idesc = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | (1u << 15) |
                                   (static_cast<uint32_t>(R >> 3) << 17) | ((128u >> 4) << 24);
        const uint64_t a_desc0 = smem_desc(base, kAtom, 1024, kSwizzle128B);
        const uint64_t b_desc0 = smem_desc(base + kWBytes, 16, 1024, kSwizzle128B);
        const uint32_t tmem = __shfl_sync(0xffffffffu, C.tmem_base, 0);
        Place at;
        int seg = 0;  // accumulators
        int block = first.block;
        bool ok = true;
        for (int step = begin; step < end && ok; ++step) {
            const bool starts = step == begin || block == 0, ends = step == end - 1 || block == kblocks - 1;
            const int acc = seg & 1;
            if (starts && !pair::wait_phase_warp(&C.abort, smem_u32(&C.tempty[acc]), ((seg >> 1) & 1) ^ 1, p.status,
                                                 p.wait_limit_ns))
                break;
            const int ksteps = (min(kBK, K - block * kBK) + 15) / 16;
#pragma unroll
            for (int m = 0; m < S::kMats; ++m) {
                if (!pair::wait_phase_warp(&C.abort, full0 + 8 * at.s, at.turn & 1, p.status, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint64_t off = static_cast<uint32_t>(at.s * S::kStage) >> 4;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        if (kk < ksteps) {
#pragma unroll
                            for (int q = 0; q < S::kParts; ++q)
                                mma_f16(tmem + acc * S::kAccCols + (S::kApart ? q : m) * R, a_desc0 + off + 128 * kk,
                                        b_desc0 + off + ((q * S::kXAtom + kk * 32) >> 4), idesc,
                                        !starts || kk > 0 || (!S::kApart && q > 0));
                        }
                    }
                    mma_commit(empty0 + 8 * at.s);
                    if (ends && m == S::kMats - 1) mma_commit(smem_u32(&C.tfull[acc]));
                }
                __syncwarp();
                at.next(stages);
            }
            if (ends) ++seg;
            if (++block == kblocks) block = 0;
        }
    } else if (warp < kEpiWarp0 + kEpiWarps) {
        // =========================================================== epilogue
        if (DOWN) pdl_wait();
        const int q = warp & 3;  // TMEM lane quarter this warp may read
        const int tid = threadIdx.x - kEpiWarp0 * 32;
        const uint32_t t_base = C.tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        float *const column = part + q * 32 + lane;
        int seg = 0;  // accumulators
        const auto filled = [&]() {
            if (!epilogue_all(pair::wait_phase_warp(&C.abort, smem_u32(&C.tfull[seg & 1]), (seg >> 1) & 1, p.status,
                                                    p.wait_limit_ns)))
                return false;
            tc_fence_after_sync();
            return true;
        };
        const auto released = [&]() {  // an accumulator has been read
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&C.tempty[seg & 1]));
            ++seg;
        };
        // The sums of a CTA's share of a job: its first (begun by a CTA before it) or its last one.
        const size_t slot = static_cast<size_t>(T) * S::kMats * 128;
        const auto share_of = [&](int cta, int owner) { return p.sums + (2 * static_cast<size_t>(cta) + (cta == owner)) * slot; };
        // Whether this CTA is the last of a job's to have stored its share; all of the epilogue calls it.
        const auto last_of = [&](int owner, int count) {
            __threadfence();
            epilogue_sync();
            if (tid == 0) C.arrived = atomicAdd(p.arrivals + owner, 1);
            epilogue_sync();
            const bool last = C.arrived == count - 1;
            if (last) __threadfence();
            return last;
        };
        Cursor c = first;
        for (int step = begin; step < end;) {
            const int job_begin = c.job * length, job_end = job_begin + length;
            const bool whole = step == job_begin && end >= job_end;
            const int owner = whole ? me : owner_of(job_begin), count = whole ? 1 : owner_of(job_end - 1) - owner + 1;
            float *const share = share_of(me, owner) + q * 32 + lane;
            const int col0 = col_of(c.job);
            bool ok = true;
            if constexpr (!DOWN) {
                // A thread has a column of Wg's and of Wu's product: a row's value is its own.
                const MoeUnit w = plan.unit[c.unit];
                const int col = col0 + q * 32 + lane;
                const auto finish = [&](int r, float gate, float up) {
                    if (col >= cols) return;
                    float f, unused;
                    a2av::split(mul2(act_value<ACT>(pair_of(gate, 0.0f)), pair_of(up, 0.0f)), f, unused);
                    uint32_t h, l;
                    value_parts<BF16>(f, h, l);
                    uint16_t *to = static_cast<uint16_t *>(p.h) + static_cast<size_t>(w.first + r) * p.N + col;
                    to[0] = static_cast<uint16_t>(h);
                    to[static_cast<size_t>(T) * topk * p.N] = static_cast<uint16_t>(l);
                };
                if (!filled()) break;
                for (int g = 0; g < w.rows; g += kGroup) {
                    uint32_t v[kGroup][2] = {};
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) {
                        if (g + i < w.rows) {
                            const uint32_t at = t_base + (seg & 1) * S::kAccCols + plan.pairs[w.first + g + i] / topk;
                            tmem_ld1(at, v[i][0]);
                            tmem_ld1(at + R, v[i][1]);
                        }
                    }
                    tmem_ld1_wait(v);
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) {
                        if (g + i < w.rows) {
                            const float gate = __uint_as_float(v[i][0]), up = __uint_as_float(v[i][1]);
                            if (whole) {
                                finish(g + i, gate, up);
                            } else {
                                share[(g + i) * 256] = gate;
                                share[(g + i) * 256 + 128] = up;
                            }
                        }
                    }
                }
                released();
                if (!whole && last_of(owner, count)) {
                    // Four shares (of G rows) are asked for together, and added in order.
                    constexpr int G = R == 16 ? 1 : 4;
                    for (int r = 0; r < w.rows; r += G) {
                        float gate[G] = {}, up[G] = {};
                        for (int k = 0; k < count; k += 4) {
                            float a[4][G], b[4][G];
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const float *at = share_of(owner + min(k + h, count - 1), owner) + q * 32 + lane + r * 256;
#pragma unroll
                                for (int g = 0; g < G; ++g) {
                                    const bool there = k + h < count && r + g < w.rows;
                                    a[h][g] = there ? __ldcg(at + g * 256) : 0.0f;
                                    b[h][g] = there ? __ldcg(at + g * 256 + 128) : 0.0f;
                                }
                            }
#pragma unroll
                            for (int h = 0; h < 4; ++h)
#pragma unroll
                                for (int g = 0; g < G; ++g) gate[g] += a[h][g], up[g] += b[h][g];
                        }
#pragma unroll
                        for (int g = 0; g < G; ++g)
                            if (r + g < w.rows) finish(r + g, gate[g], up[g]);
                    }
                }
                c.unit = ++c.job / strips;
                step = min(end, job_end);
            } else {
                for (int t = 0; t < T; ++t) column[t * 128] = 0.0f;
                for (const int until = min(end, job_end); step < until;) {
                    if (!(ok = filled())) break;
                    const MoeUnit w = plan.unit[c.unit];
#pragma unroll
                    for (int g = 0; g < R; g += 16) {
                        if (g < w.rows) {
                            uint32_t r[16], low[16];
                            tmem_ld16(t_base + (seg & 1) * S::kAccCols + g, r);
                            if constexpr (S::kApart) {
                                tmem_ld16(t_base + (seg & 1) * S::kAccCols + R + g, low);
                                tmem_ld16_wait(low);
                            }
                            tmem_ld16_wait(r);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                if (g + i < w.rows) {
                                    const int pair = plan.pairs[w.first + g + i];
                                    float *to = column + pair / topk * 128;
                                    float d = __uint_as_float(r[i]);
                                    if constexpr (S::kApart) d = sum_of_parts(d, __uint_as_float(low[i]));
                                    *to = fmaf(plan.weight[pair], d, *to);
                                }
                            }
                        }
                    }
                    released();
                    step = min(until, step - c.block + kblocks);
                    c.block = 0;
                    if (++c.unit == units) c.unit = 0, ++c.job;
                }
                if (!ok) break;
                bool mine = whole;
                if (whole) {
                    epilogue_sync();
                } else {
                    for (int t = 0; t < T; ++t) share[t * 128] = column[t * 128];
                    mine = !p.joined && last_of(owner, count);
                }
                // Four columns of a row, from their sums.
                const auto finish = [&](int i, f32x2 lo, f32x2 hi) {
                    const int r = i / 32, col = i % 32 * 4;
                    if (col0 + col >= cols) return;
                    const size_t o = static_cast<size_t>(r) * p.H + col0 + col;
                    if (p.residual) {
                        const uint2 res = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.residual) + o);
                        lo = add2(lo, unpack2<BF16>(res.x));
                        hi = add2(hi, unpack2<BF16>(res.y));
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + o) = make_uint2(pack2<BF16>(lo), pack2<BF16>(hi));
                };
                constexpr int kAll = kEpiWarps * 32;
                if (whole) {
                    for (int i = tid; i < T * 32; i += kAll) {
                        const float4 b = reinterpret_cast<const float4 *>(part)[i];
                        finish(i, pair_of(b.x, b.y), pair_of(b.z, b.w));
                    }
                } else if (mine) {
                    // (as above)
                    for (int i = tid; i < T * 32; i += kAll) {
                        f32x2 lo = 0, hi = 0;
                        for (int k = 0; k < count; k += 4) {
                            float4 v[4];
#pragma unroll
                            for (int h = 0; h < 4; ++h)
                                v[h] = k + h < count ? __ldcg(reinterpret_cast<const float4 *>(share_of(owner + k + h, owner)) + i)
                                                     : make_float4(0, 0, 0, 0);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                lo = add2(lo, pair_of(v[h].x, v[h].y));
                                hi = add2(hi, pair_of(v[h].z, v[h].w));
                            }
                        }
                        finish(i, lo, hi);
                    }
                }
                epilogue_sync();  // the sums have been read
            }
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(C.tmem_base, S::kTmemCols);
    }
}

// y from the shares of the second kernel's jobs, four columns of a row a thread: all
// of the GPU reads them at once, where the last CTA of a job would take a
// microsecond for every 14 KB.
constexpr int kJoinThreads = 128;
template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) moe_join_kernel(const MoeRowsLaunch p) {
    const int vec = blockIdx.x * kJoinThreads + threadIdx.x, row = blockIdx.y, job = vec / 32;
    const size_t o = static_cast<size_t>(row) * (p.H / 4) + vec;  // of four columns
    pdl_trigger();
    pdl_wait();
    if (4 * vec >= p.H) return;
    const int units = *p.units, kblocks = (p.N + kBK - 1) / kBK, strips = (p.H + 127) / 128;
    const int ctas = moe_ctas<true>(p.choice, kMoeCtas, units, strips, kblocks);
    const int64_t length = static_cast<int64_t>(units) * kblocks, total = length * strips;
    const auto owner_of = [&](int64_t step) { return static_cast<int>(((step + 1) * ctas - 1) / total); };
    const int owner = owner_of(job * length), count = owner_of((job + 1) * length - 1) - owner + 1;
    if (count == 1) return;  // (stored where it was made)
    const size_t slot = static_cast<size_t>(p.choice.T) * 32;
    const float4 *at = reinterpret_cast<const float4 *>(p.sums) + (2 * static_cast<size_t>(owner) + 1) * slot +
                       static_cast<size_t>(row) * 32 + vec % 32;
    f32x2 lo = 0, hi = 0;
    for (int k = 0; k < count; k += 8) {
        float4 v[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            // (the first CTA's share is its last one, the others' their first)
            const float4 *from = at + (k + h == 0 ? 0 : (2 * static_cast<size_t>(k + h) - 1) * slot);
            v[h] = k + h < count ? __ldcg(from) : make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            lo = add2(lo, pair_of(v[h].x, v[h].y));
            hi = add2(hi, pair_of(v[h].z, v[h].w));
        }
    }
    if (p.residual) {
        const uint2 res = static_cast<const uint2 *>(p.residual)[o];
        lo = add2(lo, unpack2<BF16>(res.x));
        hi = add2(hi, unpack2<BF16>(res.y));
    }
    static_cast<uint2 *>(p.y)[o] = make_uint2(pack2<BF16>(lo), pack2<BF16>(hi));
}

template <bool BF16, bool DOWN, int ACT, int R>
cudaError_t launch_rows(MoeRowsLaunch &p, cudaStream_t stream) {
    auto kern = moe_rows_kernel<BF16, DOWN, ACT, R>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    p.stages = Shape<BF16, DOWN, R>::stages(p.choice.T);
    return launch_pdl(kern, dim3(kMoeCtas), dim3(kThreads), kSmem, 0, stream, p);
}

// Rows multiplied: all tokens, or a unit's: what the fullest expert is expected to
// have, so that one pass over its weights is usual.  (Always 64, us: 8 tokens over
// 64 experts of 2048 x 1408 165 against 120; always 16 in the second kernel: 64
// tokens over 8 experts of 4096 x 4096 207 against 180.)
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
    if (bf16)
        return act == A2AV_ACT_SILU ? launch_unit<true, false, A2AV_ACT_SILU>(p, stream)
                                    : launch_unit<true, false, A2AV_ACT_GELU_TANH>(p, stream);
    return act == A2AV_ACT_SILU ? launch_unit<false, false, A2AV_ACT_SILU>(p, stream)
                                : launch_unit<false, false, A2AV_ACT_GELU_TANH>(p, stream);
}

cudaError_t launch_moe_down(MoeRowsLaunch p, bool bf16, cudaStream_t stream) {
    p.joined = p.choice.T > kAloneTokens;
    const cudaError_t err =
        bf16 ? launch_unit<true, true, A2AV_ACT_SILU>(p, stream) : launch_unit<false, true, A2AV_ACT_SILU>(p, stream);
    if (err != cudaSuccess || !p.joined) return err;
    const dim3 grid((p.H / 4 + kJoinThreads - 1) / kJoinThreads, p.choice.T);
    return launch_pdl(bf16 ? moe_join_kernel<true> : moe_join_kernel<false>, grid, kJoinThreads, 0, 0, stream, p);
}

}  // namespace a2av
