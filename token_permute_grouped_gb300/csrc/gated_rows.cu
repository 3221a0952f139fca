// The gated block for a few rows (decode and small batches): h = act(x Wg_j) *
// (x Wu_j) for the rows of each expert j that has any, straight from ataOut.
//
// Bound by the bytes of the active experts' weights, so the weights stream:
// they are the 128-row operand of tcgen05.mma (M, MN-major as they lie in
// memory) and the rows of x the narrow one (N: 16 to 128, K-major, copied
// from where they arrived by four warps; a TMA row gather brings four rows an
// instruction, and 16 a stage were slower than the weights).  A job is 64
// columns of one expert: a stage's weight tile is 128 of K x 64 columns of Wg
// as the first atom and of Wu as the second, so one MMA makes G in TMEM lanes
// 0-63 and U in lanes 64-127.  About 200 KB of stages are in flight on every
// SM, across job boundaries.
//
// There are few jobs (64 for four experts of 1024 columns), so the contraction
// of a job is split over the CTAs of a cluster, 1 to 8, whichever spreads the
// expected jobs best over the SMs.  Each CTA puts its part into its own shared
// memory, and after a barrier CTA r of S finishes the r-th of S column blocks,
// adding the S parts in order through distributed shared memory: the same sum
// every time, and nothing passes through global memory.
//
// Per CTA: warp 0 loads the weights, warp 1 issues the MMAs, warps 2-5 are the
// epilogue, warps 6-9 copy the rows of x.
// Every wait is bounded, as in the GEMMs.
//
// 8 rows over 4 experts of 4096 x 1024 (60 MB of weights where 3.6 have rows):
// 14 us a call, 4.2 TB/s with the launch, the counting and the exchange in it;
// 16 rows over 32 experts of 4096 x 1536 (about 13 have rows, 320 MB), 62 us,
// 5.2 TB/s.
#include <algorithm>
#include <cmath>

#include "activation.cuh"
#include "ffn.h"
#include "pair.cuh"
#include "pdl.cuh"
#include "per_device.h"
#include "segments.cuh"

namespace a2av {

namespace {

constexpr int kRowThreads = 10 * 32;
constexpr int kMmaWarp = 1;
constexpr int kEpiWarp0 = 2;
constexpr int kCopyWarp0 = 6;
constexpr int kCopyWarps = 4;
constexpr int kAhead = 8;                    // K blocks of a job's weights fetched before the rows are counted
constexpr int kMaxSplit = 8;                 // CTAs of a cluster
constexpr int kBK = 128;                     // contraction elements a stage
constexpr int kCols = 64;                    // output columns of a job
constexpr uint32_t kAtom = 128 * 128;        // 128 k-rows x 64 columns of weights
constexpr uint32_t kWBytes = 2 * kAtom;      // gate atom, up atom

template <int R>
struct RowShape {
    static constexpr uint32_t kXAtom = R * 128;              // R rows x 64 elements
    static constexpr uint32_t kStage = kWBytes + 2 * kXAtom;
    static constexpr int kStages = R <= 32 ? 5 : 3;
    static constexpr uint32_t kLag = kStages > 3 ? 2 : 1;    // stages whose rows of x are in flight beside the newest
    static constexpr uint32_t kPart = R * 128 * 4;           // fp32 [R][128]
    // With 128 rows the parts take the place of the stages, which then wait
    // for them between jobs (there is no room for both).
    static constexpr bool kShared = R == 128;
    static constexpr uint32_t kTmemCols = 2 * R < 32 ? 32 : 2 * R;
};

struct RowControl {
    uint64_t full[5], empty[5];
    uint64_t tfull[2], tempty[2];
    uint64_t ready;   // every CTA of the cluster has stored its rows' part
    uint64_t free;    // every CTA of the cluster has read this CTA's part
    uint32_t tmem_base;
    int32_t abort;
    int32_t n_active;
    int32_t expert[kMaxExperts];
    int32_t start[kMaxExperts + 1];  // first job of each active expert
    SegmentTable seg;
};
constexpr size_t kRowControlBytes = (sizeof(RowControl) + 1023) / 1024 * 1024;

template <int R>
constexpr size_t row_smem() {
    return 1024 + RowShape<R>::kStages * RowShape<R>::kStage + (RowShape<R>::kShared ? 0 : RowShape<R>::kPart) +
           kRowControlBytes;
}
static_assert(row_smem<16>() <= 232448 && row_smem<32>() <= 232448 && row_smem<64>() <= 232448 &&
                  row_smem<128>() <= 232448,
              "shared memory per CTA");

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

// A TMA box into L2 only.
__device__ __forceinline__ void prefetch_3d(const void *tmap, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

struct Job {
    int expert, col0, first;  // local expert, first column, first of its rows
};
__device__ __forceinline__ Job job_at(const RowControl &c, int job, int W, int rows_per_pass) {
    int a = 0;
    while (job >= c.start[a + 1]) ++a;
    const int j = c.expert[a];
    const int rows = c.seg.dst[(j + 1) * W] - c.seg.dst[j * W];
    const int passes = (rows + rows_per_pass - 1) / rows_per_pass;
    const int local = job - c.start[a];
    return {j, local / passes * kCols, local % passes * rows_per_pass};
}

template <bool BF16, int ACT, int R>
__global__ void __launch_bounds__(kRowThreads, 1) gated_rows_kernel(const __grid_constant__ GatedRowsLaunch p) {
    using S = RowShape<R>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    float *part = reinterpret_cast<float *>(base_ptr + (S::kShared ? 0 : S::kStages * S::kStage));
    RowControl &C =
        *reinterpret_cast<RowControl *>(base_ptr + S::kStages * S::kStage + (S::kShared ? 0 : S::kPart));

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int split = p.split;  // CTAs of a cluster
    const int rank = static_cast<int>(pair::cluster_rank());
    const int strips = (p.N + kCols - 1) / kCols;
    if (warp == 0) {
        // (The kernel that stages the rows let this one start after all before it had
        // completed, and nothing that it writes is read here.)
        if (!p.after_permute) pdl_wait();
        const bool good = build_segments(p.recvCounts, p.W, p.e, p.A, C.seg, lane);
        int rows = 0;
        if (lane < p.e && good) rows = C.seg.dst[(lane + 1) * p.W] - C.seg.dst[lane * p.W];
        const int jobs = (rows + R - 1) / R * strips;
        int inc = jobs;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, rows > 0);
        const int slot = __popc(mask & ((1u << lane) - 1u));
        if (rows > 0) {
            C.expert[slot] = lane;
            C.start[slot] = inc - jobs;
        }
        if (lane == 31) C.start[__popc(mask)] = inc;
        if (lane == 0) {
            C.n_active = __popc(mask);
            C.abort = 0;
            if (blockIdx.x == 0) {
                if (!p.after_permute) *p.status = good ? 0 : kStatusBadCounts;
                else if (!good) atomicOr(p.status, kStatusBadCounts);
            }
        }
    } else if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&C.tmem_base), S::kTmemCols);
        tmem_relinquish();
    } else if (warp == kEpiWarp0) {
        if (lane == 0) {
            for (int s = 0; s < S::kStages; ++s) {
                mbar_init(smem_u32(&C.full[s]), 1 + kCopyWarps);
                mbar_init(smem_u32(&C.empty[s]), 1);
            }
            for (int a = 0; a < 2; ++a) {
                mbar_init(smem_u32(&C.tfull[a]), 1);
                mbar_init(smem_u32(&C.tempty[a]), 4);
            }
            mbar_init(smem_u32(&C.ready), 4 * split);
            mbar_init(smem_u32(&C.free), 4 * split);
            fence_barrier_init();
        }
    } else if (warp == kEpiWarp0 + 1 && lane == 0) {
        prefetch_tensormap(&p.tmGate);
        prefetch_tensormap(&p.tmUp);
        // With rows for nearly every expert, this CTA's first job is known
        // before they are counted, and while the kernel before this one ends:
        // its weights may be on their way to L2.
        const int job = blockIdx.x / split, kblocks = (p.K + kBK - 1) / kBK;
        const int kb0 = kblocks * rank / split, kb1 = kblocks * (rank + 1) / split;
        if (job < p.guess * strips)
            for (int kb = kb0; kb < min(kb1, kb0 + kAhead); ++kb) {
                prefetch_3d(&p.tmGate, job % strips * kCols, kb * kBK, job / strips);
                prefetch_3d(&p.tmUp, job % strips * kCols, kb * kBK, job / strips);
            }
    }
    tc_fence_before_sync();
    pair::sync_all();
    tc_fence_after_sync();

    const int total = C.start[C.n_active];
    const int cluster = blockIdx.x / split, clusters = gridDim.x / split;
    const int kblocks = (p.K + kBK - 1) / kBK;
    const int kb0 = kblocks * rank / split, kb1 = kblocks * (rank + 1) / split;  // this CTA's part
    const uint32_t full0 = smem_u32(&C.full[0]), empty0 = smem_u32(&C.empty[0]);
    const uint32_t ready = smem_u32(&C.ready), freed = smem_u32(&C.free);
    // Before the stages of a CTA's job number jl are filled, the parts of the job
    // before it have been read, where they share the memory.
    const auto stages_free = [&](uint32_t jl, auto wait) {
        return !S::kShared || jl == 0 || wait(&C.abort, freed, (jl - 1) & 1, p.status, p.wait_limit_ns);
    };

    if (warp == 0) {
        // ================================================== producer (weights)
        if (lane == 0) {
            uint32_t it = 0, jl = 0;
            bool ok = true;
            for (int job = cluster; job < total && ok; job += clusters, ++jl) {
                const Job w = job_at(C, job, p.W, R);
                ok = stages_free(jl, pair::wait_phase);
                if (!ok) break;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % S::kStages;
                    if (!pair::wait_phase(&C.abort, empty0 + 8 * s, ((it / S::kStages) & 1) ^ 1, p.status,
                                          p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = base + s * S::kStage, bar = full0 + 8 * s;
                    mbar_arrive_expect_tx(bar, kWBytes);
                    tma_load_3d(st, &p.tmGate, bar, w.col0, kb * kBK, w.expert);
                    tma_load_3d(st + kAtom, &p.tmUp, bar, w.col0, kb * kBK, w.expert);
                }
            }
            pdl_trigger();
            if (p.after_permute) pdl_wait();
            for (int i = 0; i < S::kStages && ok; ++i, ++it)
                ok = pair::wait_phase(&C.abort, empty0 + 8 * (it % S::kStages), ((it / S::kStages) & 1) ^ 1, p.status,
                                      p.wait_limit_ns);
            if (!ok) pair::let_settle();
        }
    } else if (warp >= kCopyWarp0) {
        // ================================================== producer (rows of x)
        // A thread copies the same 16-byte piece of a stage's 256 bytes of every
        // eighth row.  The copies are generic-proxy writes, so a stage is handed
        // to the MMA by this thread's fence once they have landed: S::kLag stages
        // later, or as soon as there is no stage to fill.
        const int ct = threadIdx.x - kCopyWarp0 * 32, piece = ct % 16, r0 = ct / 16;
        const uint32_t to = (piece / 8) * S::kXAtom + r0 * 128 + (((piece % 8) ^ (r0 & 7)) << 4);
        uint32_t it = 0, given = 0, jl = 0;  // stages issued, stages handed over, jobs
        bool ok = true;
        const auto hand_over = [&](uint32_t until) {
            fence_proxy_async_smem();
            __syncwarp();
            for (; given < until; ++given)
                if (lane == 0) mbar_arrive(full0 + 8 * (given % S::kStages));
        };
        for (int job = cluster; job < total && ok; job += clusters, ++jl) {
            const Job w = job_at(C, job, p.W, R);
            if (S::kShared) {  // (nothing of this job can be read before the parts are gone)
                cp_async_wait<0>();
                hand_over(it);
            }
            ok = stages_free(jl, pair::wait_phase_warp);
            if (!ok) break;
            __syncwarp();
            const int row0 = C.seg.dst[w.expert * p.W], rows = C.seg.dst[(w.expert + 1) * p.W] - row0;
            const uint16_t *src[R / 8];
#pragma unroll
            for (int i = 0; i < R / 8; ++i) {
                const int r = w.first + r0 + 8 * i;
                src[i] = nullptr;  // no such row: zeros
                if (r < rows)
                    src[i] = static_cast<const uint16_t *>(p.x) +
                             static_cast<size_t>(source_row(C.seg, p.W, p.e, row0 + r)) * p.K + piece * 8;
            }
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % S::kStages;
                const uint32_t par = ((it / S::kStages) & 1) ^ 1;
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
                const bool in_k = kb * kBK + piece * 8 < p.K;
#pragma unroll
                for (int i = 0; i < R / 8; ++i) {
                    const bool live = in_k && src[i] != nullptr;
                    cp_async_16_or_zero(x_st + i * 1024, live ? src[i] + kb * kBK : static_cast<const uint16_t *>(p.x),
                                        live ? 16 : 0);
                }
                cp_async_commit();
                if (it - given >= S::kLag) {
                    cp_async_wait<S::kLag>();
                    hand_over(it + 1 - S::kLag);
                }
            }
        }
        cp_async_wait<0>();
        if (ok) hand_over(it);
    } else if (warp == kMmaWarp) {
        // =========================================================== MMA issuer
        if (lane == 0) {
            // A: the weights, MN-major (atoms of 64 columns 16 KB apart, 8-row K groups 1024 B apart, a K step
            // of 16 rows 2 KB).  B: x, K-major (8-row groups 1024 B apart, a K step of 16 elements 32 B).
            constexpr uint32_t idesc = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | (1u << 15) |
                                       (static_cast<uint32_t>(R >> 3) << 17) | ((128u >> 4) << 24);
            const uint64_t a_desc0 = smem_desc(base, kAtom, 1024, kSwizzle128B);
            const uint64_t b_desc0 = smem_desc(base + kWBytes, 16, 1024, kSwizzle128B);
            uint32_t it = 0, jl = 0;
            bool ok = true;
            for (int job = cluster; job < total && ok; job += clusters, ++jl) {
                const int acc = jl & 1;
                if (!pair::wait_phase(&C.abort, smem_u32(&C.tempty[acc]), ((jl >> 1) & 1) ^ 1, p.status,
                                      p.wait_limit_ns))
                    break;
                tc_fence_after_sync();
                const uint32_t d_tmem = C.tmem_base + acc * R;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % S::kStages;
                    const uint32_t par = (it / S::kStages) & 1;
                    if (!mbar_try_wait(full0 + 8 * s, par) &&
                        !pair::wait_phase(&C.abort, full0 + 8 * s, par, p.status, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint64_t ad = a_desc0 + ((s * S::kStage) >> 4), bd = b_desc0 + ((s * S::kStage) >> 4);
                    const int ksteps = (min(kBK, p.K - kb * kBK) + 15) / 16;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        if (kk < ksteps)
                            mma_f16(d_tmem, ad + 128 * kk, bd + (((kk >> 2) * S::kXAtom + (kk & 3) * 32) >> 4), idesc,
                                    kb > kb0 || kk > 0);
                    mma_commit(empty0 + 8 * s);
                }
                if (ok) mma_commit(smem_u32(&C.tfull[acc]));
            }
        }
    } else {
        // =========================================================== epilogue
        const int q = warp & 3;  // TMEM lane quarter this warp may read
        const int tid = threadIdx.x - kEpiWarp0 * 32;
        const int own = kCols / split;  // columns this CTA finishes
        uint32_t jl = 0;
        for (int job = cluster; job < total; job += clusters, ++jl) {
            const Job w = job_at(C, job, p.W, R);
            const int row0 = C.seg.dst[w.expert * p.W], rows = C.seg.dst[(w.expert + 1) * p.W] - row0;
            const int live = min(R, rows - w.first);
            const int acc = jl & 1;
            if (!pair::wait_phase_warp(&C.abort, smem_u32(&C.tfull[acc]), (jl >> 1) & 1, p.status, p.wait_limit_ns)) break;
            tc_fence_after_sync();
            const uint32_t t_base = C.tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * R;
            if (!pair::wait_phase_warp(&C.abort, freed, (jl & 1) ^ 1, p.status, p.wait_limit_ns)) break;
#pragma unroll
            for (int c = 0; c < R; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(t_base + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    part[(c + i) * 128 + q * 32 + lane] = kb1 > kb0 ? __uint_as_float(r[i]) : 0.0f;
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&C.tempty[acc]));
                for (int c = 0; c < split; ++c) pair::arrive_cluster(pair::map_to_rank(ready, c));
            }
            if (!pair::wait_phase_warp(&C.abort, ready, jl & 1, p.status, p.wait_limit_ns)) break;
            for (int i = tid; i < live * own / 4; i += 4 * 32) {
                const int r = i / (own / 4), c = rank * own + i % (own / 4) * 4;
                if (w.col0 + c < p.N) {  // (N is a multiple of 8: all four columns or none)
                    const uint32_t at = smem_u32(part + r * 128 + c);
                    float4 g[kMaxSplit], u[kMaxSplit];
#pragma unroll
                    for (int k = 0; k < kMaxSplit; ++k) {
                        if (k < split) {
                            const uint32_t a = pair::map_to_rank(at, k);
                            g[k] = ld_cluster_f32x4(a);
                            u[k] = ld_cluster_f32x4(a + kCols * 4);
                        }
                    }
#pragma unroll
                    for (int k = 1; k < kMaxSplit; ++k) {
                        if (k < split) {
                            g[0] = make_float4(g[0].x + g[k].x, g[0].y + g[k].y, g[0].z + g[k].z, g[0].w + g[k].w);
                            u[0] = make_float4(u[0].x + u[k].x, u[0].y + u[k].y, u[0].z + u[k].z, u[0].w + u[k].w);
                        }
                    }
                    const size_t o = static_cast<size_t>(row0 + w.first + r) * p.N + w.col0 + c;
                    if (p.saved[0]) {
                        *reinterpret_cast<float4 *>(p.saved[0] + o) = g[0];
                        *reinterpret_cast<float4 *>(p.saved[1] + o) = u[0];
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.h) + o) = make_uint2(
                        pack2<BF16>(mul2(act_value<ACT>(pair_of(g[0].x, g[0].y)), pair_of(u[0].x, u[0].y))),
                        pack2<BF16>(mul2(act_value<ACT>(pair_of(g[0].z, g[0].w)), pair_of(u[0].z, u[0].w))));
                }
            }
            if (S::kShared) fence_proxy_async_smem();  // TMA writes over the part next
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

// What a job costs beside its K blocks, in K blocks (16 rows over 32 experts of
// 4096 x 1536: 62 us with 2 to 4, 76 with 0 or 1).
constexpr double kJobCost = 3.0;

// Clusters of 1, 2, 4 and 8 CTAs resident at once.
struct Resident {
    int clusters[4];
};
template <int R>
const Resident *resident_clusters() {
    static PerDevice<Resident> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
    return cache.get(dev, [](Resident &r) {
        for (int i = 0; i < 4; ++i)
            r.clusters[i] = max_clusters(gated_rows_kernel<true, A2AV_ACT_SILU, R>, kRowThreads, row_smem<R>(), 1 << i);
        return r.clusters[0] > 0;
    });
}

template <bool BF16, int ACT, int R>
cudaError_t launch_rows(GatedRowsLaunch &p, cudaStream_t stream) {
    auto kern = gated_rows_kernel<BF16, ACT, R>;
    constexpr size_t smem = row_smem<R>();
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    const Resident *of_device = resident_clusters<R>();
    if (!of_device) return cudaErrorUnknown;
    const int(&resident)[4] = of_device->clusters;
    // The split of K that takes the least time, counted in K blocks a CTA
    // streams plus what a job costs beside them, for the experts that rows
    // spread at random would reach.
    const double reached = p.e * (1.0 - std::pow(1.0 - 1.0 / p.e, static_cast<double>(p.A)));
    const int strips = (p.N + kCols - 1) / kCols;
    const double jobs = std::ceil(reached - 0.5) * strips;
    // Weights fetched before the rows are counted, where most experts will have some
    // (us, without / with; share reached): 4 experts of 4096 x 1024, 8 rows (0.90)
    // 15.7 / 14.7, 32 (1.00) 15.8 / 15.2; 16 experts, 32 rows (0.87) 37.8 / 36.9.
    // Below, some of what is fetched is not used: 16 rows (0.64) 39.3 / 39.3.
    p.guess = reached > 0.85 * p.e ? p.e : 0;
    const int kblocks = (p.K + kBK - 1) / kBK;
    double best = 0.0;
    for (int i = 0; i < 4; ++i) {
        if (resident[i] <= 0) continue;
        const double rounds = std::ceil(jobs / resident[i]);
        const double cost = rounds * (std::ceil(static_cast<double>(kblocks) / (1 << i)) + kJobCost);
        if (i == 0 || cost < best) {
            best = cost;
            p.split = 1 << i;
            p.grid = resident[i] << i;
        }
    }
    const int64_t most_jobs = (static_cast<int64_t>(std::min(p.e, p.A)) + p.A / R) * strips;
    p.grid = static_cast<int>(std::min<int64_t>(p.grid, most_jobs * p.split));
    return launch_pdl(kern, dim3(p.grid), dim3(kRowThreads), smem, p.split, stream, p);
}

template <bool BF16, int ACT>
cudaError_t launch_rows_tile(GatedRowsLaunch &p, cudaStream_t stream) {
    const double most = gated_rows_most(p.A, p.e);  // so that one pass over the weights is usual
    if (most <= 16) return launch_rows<BF16, ACT, 16>(p, stream);
    if (most <= 32) return launch_rows<BF16, ACT, 32>(p, stream);
    // 128 rows a pass where that one is usual, or where one expert has up to two
    // (256 rows of 7168 x 2048: 31.8 us).
    if (most > 64) return launch_rows<BF16, ACT, 128>(p, stream);
    return launch_rows<BF16, ACT, 64>(p, stream);
}

}  // namespace

double gated_rows_most(int64_t A, int32_t e) {  // the mean and three deviations
    const double mean = static_cast<double>(A) / e;
    return std::min<double>(static_cast<double>(A), mean + 3.0 * std::sqrt(mean) + 1.0);
}

cudaError_t launch_gated_rows(GatedRowsLaunch p, bool bf16, int act, cudaStream_t stream) {
    if (bf16)
        return act == A2AV_ACT_SILU ? launch_rows_tile<true, A2AV_ACT_SILU>(p, stream)
                                    : launch_rows_tile<true, A2AV_ACT_GELU_TANH>(p, stream);
    return act == A2AV_ACT_SILU ? launch_rows_tile<false, A2AV_ACT_SILU>(p, stream)
                                : launch_rows_tile<false, A2AV_ACT_GELU_TANH>(p, stream);
}

}  // namespace a2av
