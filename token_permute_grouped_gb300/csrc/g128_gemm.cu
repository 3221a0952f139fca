// Grouped GEMM of 8-bit rows with a float32 scale per 128 codes, on tcgen05
// tensor cores (sm_103a): tiles of 256 rows x 256 columns on CTA pairs, or of 128 x
// 128 on single CTAs where there are few.
//
//   y[i][n] = sum over b of xs[i][b] ws[n / 128][b] sum over k in b of x[i][k] w[n][k]
//
// The scales are arbitrary floats, so the tensor cores cannot apply them: each
// block of 128 codes along K is a product of its own (four MMAs of K = 32 that
// start a TMEM accumulator afresh), which the epilogue warps multiply by its
// scales and add to sums in their registers while the next block is multiplied
// into another accumulator.  A lane's row has one scale and a warp's 128 columns
// one, so a block costs a lane one product and 64 packed FMAs.
//
// Per CTA: warps 0 and 2 load (a stage is one K block: 16 KB of rows, 16 KB of
// weights, 128-byte swizzle), warp 1 issues the MMAs (a pair's even CTA), warps 4-11 sum
// and store, two for each TMEM lane quarter, half of the columns each.  They take
// the registers that the first four warps leave.
// A warp that loads or issues goes along as a whole and one lane issues, which
// leaves the operands in uniform registers: a branch on the lane costs two to four
// times the slots.  Every wait is bounded, as in the other GEMMs.
//
// Bound by the scaling: a K block's 256 x 256 products cost a pair's tensor cores
// 512 clocks and each lane 64 packed FMAs, loads of the same from TMEM and a wait.
// 34,502 rows of 7168 x 4096 from 32 sources take 717 to 856 us (2.4 to 2.8
// PFLOP/s, the power limit in force), 56 of them the copying of rows; the product
// with scales in the tensor cores (a2av_gmm_mx_run) takes 650 to 700 for the shape.
#include <algorithm>

#include "activation.cuh"
#include "g128.h"
#include "pair.cuh"
#include "pdl.cuh"
#include "segments.cuh"

namespace a2av {

namespace {

constexpr int BM = 128;             // rows of a CTA
constexpr int BK = 128;             // codes of a K block, which has one scale
constexpr int kMmaWarp = 1;
constexpr int kLoadWarpB = 2;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
// Registers of a thread: 384 x 168 at the launch, as many after the split.
constexpr int kRegsAtLaunch = 168, kRegsFew = 56, kRegsMany = 224;
static_assert(kEpiWarp0 * kRegsFew + kEpiWarps * kRegsMany <= (kEpiWarp0 + kEpiWarps) * kRegsAtLaunch, "registers of a CTA");
constexpr uint32_t kTmemCols = 512;

constexpr int kStages = 6;
constexpr uint32_t kA = BM * BK, kB = 128 * BK, kStageBytes = kA + kB;

template <bool PAIR>
struct Shape {
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int M = kCtas * BM, N = kCtas * 128;  // of a tile
    static constexpr int kAccs = kTmemCols / N;            // accumulators
    static constexpr int kCols = N / 2;                    // columns of an epilogue warp
};

constexpr uint32_t kTurnBytes = 32 * 64;  // of an epilogue warp: 32 x 32 results

struct Group {
    int32_t row0, rows, tile_start;
};
struct Control {
    uint64_t full[kStages], empty[kStages];
    uint64_t tfull[4], tempty[4];
    uint32_t tmem_base;
    int32_t abort;
    int32_t total_tiles;
    Group g[kMaxExperts + 1];
    SegmentTable seg;
};
constexpr size_t kControlBytes = (sizeof(Control) + 1023) / 1024 * 1024;

constexpr size_t kSmem = 1024 + kStages * kStageBytes + kEpiWarps * kTurnBytes + kControlBytes;
static_assert(kSmem <= 232448, "shared memory per CTA");

struct Tile {
    int g, m, n;
};
__device__ __forceinline__ Tile tile_at(const Control &c, int t, int tn) {
    int g = 0;
    while (t >= c.g[g + 1].tile_start) ++g;
    const int local = t - c.g[g].tile_start;
    return {g, local / tn, local % tn};
}

// kind::f8f6f4: fp32 accumulator, both operands of one 8-bit format (0 E4M3, 1
// E5M2) and K-major, M x N.
__device__ __forceinline__ uint32_t instr_desc_f8(uint32_t qtype, uint32_t M, uint32_t N) {
    return (1u << 4) | (qtype << 7) | (qtype << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

template <bool PAIR>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// The barrier of a tile's CTAs.
template <bool PAIR>
__device__ __forceinline__ void sync_tile() {
    if constexpr (PAIR) pair::sync_all();
    else __syncthreads();
}

// A warp's bounded wait, in line (a call would put an epilogue's sums aside, and
// does not fit the split of registers), with one answer for the warp.
__device__ __forceinline__ bool wait_in_line(int32_t *abort_flag, uint32_t bar, uint32_t parity, int32_t *status,
                                             uint64_t limit_ns) {
    bool ok = pair::try_wait_cluster(bar, parity);
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        for (int i = 1; !(ok = pair::try_wait_cluster(bar, parity)); ++i) {
            if (i % 64 != 0) continue;
            if (*reinterpret_cast<volatile int32_t *>(abort_flag)) break;
            if (global_timer_ns() - t0 > limit_ns) {
                *reinterpret_cast<volatile int32_t *>(abort_flag) = 1;
                atomicOr(status, kStatusTimeout);
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

template <bool BF16, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) g128_gemm_kernel(const __grid_constant__ G128Launch p) {
    using S = Shape<PAIR>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const uint32_t turn0 = base + kStages * kStageBytes;
    Control &C = *reinterpret_cast<Control *>(base_ptr + kStages * kStageBytes + kEpiWarps * kTurnBytes);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t rank = PAIR ? pair::cluster_rank() : 0;
    const int unit = blockIdx.x / S::kCtas, nunits = gridDim.x / S::kCtas;
    const int tn = (p.N + S::N - 1) / S::N, kblocks = p.K / BK;

    if (warp == 0) {
        // (A kernel that this one overlaps has waited for all before it.)
        if (!p.after_permute) pdl_wait();
        const bool good = build_segments(p.recvCounts, p.W, p.e, p.A, C.seg, lane);
        int row0 = 0, rows = 0, tiles = 0;
        if (lane < p.e) {
            row0 = C.seg.dst[lane * p.W];
            rows = C.seg.dst[(lane + 1) * p.W] - row0;
            tiles = good ? blocks_of(rows, S::M) * tn : 0;
        }
        int inc = tiles;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane < p.e) C.g[lane] = Group{row0, rows, inc - tiles};
        if (lane == 31) {
            C.g[p.e] = Group{0, 0, inc};
            C.total_tiles = inc;
            C.abort = 0;
            if (blockIdx.x == 0) {
                if (p.write_status) *p.status = good ? 0 : kStatusBadCounts;
                else if (!good) atomicOr(p.status, kStatusBadCounts);
            }
        }
    } else if (warp == kMmaWarp) {
        if constexpr (PAIR) {
            pair::tmem_alloc_pair(smem_u32(&C.tmem_base), kTmemCols);
        } else {
            tmem_alloc(smem_u32(&C.tmem_base), kTmemCols);
            tmem_relinquish();
        }
    } else if (warp == kEpiWarp0) {
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(smem_u32(&C.full[s]), 2);
                mbar_init(smem_u32(&C.empty[s]), 1);
            }
            for (int a = 0; a < S::kAccs; ++a) {
                mbar_init(smem_u32(&C.tfull[a]), 1);
                mbar_init(smem_u32(&C.tempty[a]), S::kCtas * kEpiWarps);
            }
            fence_barrier_init();
        }
    } else if (warp == kEpiWarp0 + 1 && lane == 0) {
        prefetch_tensormap(&p.tmA);
        prefetch_tensormap(&p.tmB);
        if (p.direct_halves) prefetch_tensormap(&p.tmDirect);
    }
    tc_fence_before_sync();
    sync_tile<PAIR>();
    tc_fence_after_sync();

    const int total = __shfl_sync(0xffffffffu, C.total_tiles, 0);
    const uint32_t full0 = smem_u32(&C.full[0]), empty0 = smem_u32(&C.empty[0]);
    const uint32_t tfull0 = smem_u32(&C.tfull[0]), tempty0 = smem_u32(&C.tempty[0]);
    // A ring's place: stage (or accumulator) and how often it has been gone round.
    struct Place {
        int s = 0, turn = 0;
        __device__ __forceinline__ void next(int n) {
            if (++s == n) s = 0, ++turn;
        }
    };

    const auto give_up_registers = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew)); };
    if (warp == 0 || warp == kLoadWarpB) {
        // =========================================================== producers: rows, weights
        give_up_registers();
        const bool rows = warp == 0, leader = elect_one();
        const uint32_t bytes = rows ? kA : kB, to = base + (rows ? 0 : kA);
        Place at;
        bool ok = true, all_there = !p.after_permute || !rows;
        for (int t = unit; t < total && ok; t += nunits) {
            const Tile w = tile_at(C, t, tn);
            const CUtensorMap *map = &p.tmB;
            int y = w.n * S::N + static_cast<int>(rank) * 128, z = w.g;
            if (rows) {
                const int g_end = C.g[w.g].row0 + C.g[w.g].rows;
                // This CTA's first row; without a row of its own, any one (nothing of it is stored).
                const int from = w.m * S::M + static_cast<int>(rank) * BM;
                const bool live = from < C.g[w.g].rows;
                y = C.g[w.g].row0 + (live ? from : 0);
                z = 0;
                map = &p.tmA;
                if (p.direct_halves && live && half_in_one_segment(C.seg, p.W, p.e, y, g_end)) {
                    map = &p.tmDirect;
                    y = source_row(C.seg, p.W, p.e, y);
                } else if (!all_there) {
                    pdl_wait();
                    all_there = true;
                }
            }
            for (int kb = 0; kb < kblocks; ++kb, at.next(kStages)) {
                if (at.turn > 0 && !wait_in_line(&C.abort, empty0 + 8 * at.s, (at.turn & 1) ^ 1, p.status,
                                                          p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t own = full0 + 8 * at.s;
                if (leader) {
                    if (rank == 0) mbar_arrive_expect_tx(own, S::kCtas * bytes);
                    if constexpr (PAIR) pair::load_3d(to + at.s * kStageBytes, map, pair::map_to_rank(own, 0), kb * BK, y, z);
                    else tma_load_3d(to + at.s * kStageBytes, map, own, kb * BK, y, z);
                }
                __syncwarp();
            }
        }
        if (rows) {
            pdl_trigger();
            if (!all_there) pdl_wait();  // (a kernel's end implies that of all before it)
        }
        // The stages that were filled have been read.
        for (int i = 0; i < kStages && ok; ++i) {
            const int turns = at.s > i ? at.turn + 1 : at.turn;  // fills of stage i
            if (turns > 0)
                ok = wait_in_line(&C.abort, empty0 + 8 * i, (turns - 1) & 1, p.status, p.wait_limit_ns);
        }
        if (!ok) pair::let_settle();
    } else if (warp == kMmaWarp) {
        // =========================================================== MMA issuer
        give_up_registers();
        if (rank == 0) {
            const bool leader = elect_one();
            const uint32_t idesc = instr_desc_f8(static_cast<uint32_t>(p.qtype), S::M, S::N);
            const uint64_t a_desc0 = smem_desc(base, 16, 1024, kSwizzle128B);
            const uint64_t b_desc0 = smem_desc(base + kA, 16, 1024, kSwizzle128B);
            const uint32_t tmem = __shfl_sync(0xffffffffu, C.tmem_base, 0);
            Place at, acc;
            bool ok = true;
            for (int t = unit; t < total && ok; t += nunits) {
                for (int kb = 0; kb < kblocks; ++kb, at.next(kStages), acc.next(S::kAccs)) {
                    if (!wait_in_line(&C.abort, full0 + 8 * at.s, at.turn & 1, p.status, p.wait_limit_ns) ||
                        !wait_in_line(&C.abort, tempty0 + 8 * acc.s, (acc.turn & 1) ^ 1, p.status, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t off = static_cast<uint32_t>(at.s * kStageBytes) >> 4;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk)
                            mma_f8<PAIR>(tmem + acc.s * S::N, a_desc0 + off + 2 * kk, b_desc0 + off + 2 * kk, idesc, kk > 0);
                        if constexpr (PAIR) {
                            pair::commit(empty0 + 8 * at.s);
                            pair::commit(tfull0 + 8 * acc.s);
                        } else {
                            mma_commit(empty0 + 8 * at.s);
                            mma_commit(tfull0 + 8 * acc.s);
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp < kEpiWarp0) {
        give_up_registers();
    } else {
        // =========================================================== sums and stores
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        const int q = warp & 3;
        const int part = (warp - kEpiWarp0) / 4;  // of the columns
        const uint32_t turn = turn0 + static_cast<uint32_t>(warp - kEpiWarp0) * kTurnBytes;
        const uint32_t t_base = C.tmem_base + (static_cast<uint32_t>(q * 32) << 16) + part * S::kCols;
        const int scale_rows = (p.N + 127) / 128;  // of an expert's weights
        const float *xs = p.xs, *ws = p.ws;        // of this lane's row, of this warp's columns
        float xn[2] = {0, 0}, wn[2] = {0, 0};      // of the next K blocks
        bool valid = false;
        // The scales of a tile's first blocks, asked for ahead of the tile.
        const auto prepare = [&](int t) {
            const Tile w = tile_at(C, t, tn);
            const int r = w.m * S::M + static_cast<int>(rank) * BM + q * 32 + lane;
            valid = r < C.g[w.g].rows;
            const int src = valid ? source_row(C.seg, p.W, p.e, C.g[w.g].row0 + r) : 0;
            xs = p.xs + static_cast<size_t>(src) * kblocks;
            const int block = min((w.n * S::N + part * S::kCols) / 128, scale_rows - 1);
            ws = p.ws + (static_cast<size_t>(w.g) * scale_rows + block) * kblocks;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i < kblocks) {
                    xn[i] = xs[i];
                    wn[i] = ws[i];
                }
            }
        };
        Place acc;
        bool ok = true;
        if (unit < total) prepare(unit);
        for (int t = unit; t < total && ok; t += nunits) {
            f32x2 sum[S::kCols / 2];
#pragma unroll
            for (int j = 0; j < S::kCols / 2; ++j) sum[j] = 0;
            const bool row_valid = valid;
            for (int kb = 0; kb < kblocks; ++kb, acc.next(S::kAccs)) {
                const f32x2 scale = both(xn[0] * wn[0]);
                xn[0] = xn[1];
                wn[0] = wn[1];
                if (kb + 2 < kblocks) {
                    xn[1] = xs[kb + 2];
                    wn[1] = ws[kb + 2];
                }
                const uint32_t from = t_base + acc.s * S::N, empty = PAIR ? pair::map_to_rank(tempty0 + 8 * acc.s, 0) : tempty0 + 8 * acc.s;
                if (!wait_in_line(&C.abort, tfull0 + 8 * acc.s, acc.turn & 1, p.status, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                uint32_t r[2][16];
                tmem_ld16(from, r[0]);
#pragma unroll
                for (int c = 0; c < S::kCols / 16; ++c) {
                    tmem_ld16_wait(r[c & 1]);
                    if (c + 1 < S::kCols / 16) {
                        tmem_ld16(from + 16 * (c + 1), r[(c + 1) & 1]);
                    } else {  // all of it is in registers
                        tc_fence_before_sync();
                        if (lane == 0) pair::arrive_reads_done(empty);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum[8 * c + j] = fma2(pair_of(__uint_as_float(r[c & 1][2 * j]), __uint_as_float(r[c & 1][2 * j + 1])),
                                              scale, sum[8 * c + j]);
                }
            }
            if (!ok) break;
            const Tile w = tile_at(C, t, tn);
            const int row0 = C.g[w.g].row0 + w.m * S::M + static_cast<int>(rank) * BM + q * 32;
            const int rows = __popc(__ballot_sync(0xffffffffu, row_valid));  // (the first of the 32)
            const int col0 = w.n * S::N + part * S::kCols;
            if (t + nunits < total) prepare(t + nunits);
            // Each 32 x 32 block is turned around in this warp's 2 KB (64-byte rows, the
            // 16-byte chunk index XORed with (row / 2) % 4), so that a store takes 64 bytes
            // of eight rows, not 16 of 32: the next blocks' MMAs wait for these.
#pragma unroll
            for (int i = 0; i < S::kCols / 32; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2(&v)[4] = *reinterpret_cast<const f32x2(*)[4]>(&sum[16 * i + 4 * j]);
                    st_shared_v4(turn + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), pack8<BF16>(v));
                }
                __syncwarp();
                const int j = lane & 3, col = col0 + 32 * i + 8 * j;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 8 * k + (lane >> 2);
                    const uint4 v = ld_shared_v4(turn + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
                    if (r < rows && col < p.N)
                        st_stream_v4(static_cast<uint16_t *>(p.y) + static_cast<size_t>(row0 + r) * p.N + col, v);
                }
                __syncwarp();
            }
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    sync_tile<PAIR>();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        if constexpr (PAIR) pair::tmem_free_pair(C.tmem_base, kTmemCols);
        else tmem_dealloc(C.tmem_base, kTmemCols);
    }
}

template <bool BF16, bool PAIR>
cudaError_t launch_shape(const G128Launch &p, cudaStream_t stream) {
    auto kern = g128_gemm_kernel<BF16, PAIR>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, p.grid, kThreads, kSmem, PAIR ? 2 : 0, stream, p);
}

}  // namespace

cudaError_t launch_g128_gemm(const G128Launch &p, bool bf16, cudaStream_t stream) {
    if (p.pair) return bf16 ? launch_shape<true, true>(p, stream) : launch_shape<false, true>(p, stream);
    return bf16 ? launch_shape<true, false>(p, stream) : launch_shape<false, false>(p, stream);
}

// (Nearly all of an SM's shared memory: one CTA an SM.)
int g128_gemm_max_clusters() { return max_clusters(g128_gemm_kernel<true, true>, kThreads, kSmem, 2); }

}  // namespace a2av
