// Persistent ragged GEMMs of an expert layer's gated block and gradients, on
// tcgen05 tensor cores (sm_103a), for the experts j of a rank:
//
//   gated      h = act(X Wg_j) * (X Wu_j)
//   gradients  dX = D_0 W_0j^T (+ D_1 W_1j^T)  and  dW_j = X_j^T D_j
//
// Three ways of walking the operands, two kernels: both gradients' tiles are
// one list, so that they share a launch and its tail.  A cluster of two CTAs
// computes a tile of 256 rows x 256 accumulator columns with one cta_group::2
// MMA: each CTA stages 128 of the rows of A and half of the columns of B.  The
// even CTA issues the MMAs; each CTA holds its 128 rows of the accumulator.
// Where that leaves too few tiles for the SMs, tiles are half as wide (BN 128).
//
// The gated tile is BN / 2 output columns: the even CTA stages them from Wg, the
// odd one from Wu, so the accumulator's first half is G and its second U for
// the same rows and columns, and the epilogue forms act(G) * U lane by lane
// before anything is written.  The same split gives both weights' gradients
// of a gated block from one read of X.
//
// Every operand tile has one shape in shared memory: 128 rows of 128 elements,
// as two 64-element atoms of 128-byte swizzled rows (32 KB), loaded by one
// TMA box (two where the width is no multiple of 64; columns and rows past
// the tensor's end arrive as zeros).  What differs is how the tensor core
// reads it: with the contraction along the elements (K-major) or along the
// rows (MN-major), a bit in the instruction descriptor and two strides.
//
//   tile              A (rows x elements)        B (rows x elements)
//   gated             X: rows x K    K-major     W: K x columns        MN-major
//   rows' gradient    D: rows x K    K-major     W: out columns x K    K-major
//   weights' gradient X: K x M       MN-major    D: K x columns        MN-major
//
// A D_p may come as two summands of the element type; the second
// ones are further products into the same accumulator.
//
// In the weights' gradient K runs over an expert's rows, whose last block is
// ragged, and the rows behind it belong to the next expert.  That block goes
// first in each tile, is multiplied only up to its last 16 rows, and the rows
// of those that are not the expert's are overwritten with zeros in both
// operands by a warp of each CTA before the MMA may read them: multiplying by
// zero on one side alone would let another expert's infinities through.
//
// Where the gradients' tiles are few, or some far longer than the rest, their
// contraction is cut into slices, each a tile of its own whose fp32 sums go to
// the workspace; a second kernel adds them in order.
//
// A gated block's D_p may still be in the making when this kernel starts: the
// kernel before it (glu_grad.cu) writes them in the order the tiles go and
// counts the finished pieces of each 128 rows, and the producer waits for a
// tile's counts.
//
// Per CTA: warp 0 loads, warp 1 clears ragged rows (weights' gradient), warp 4
// allocates TMEM and (even CTA) issues, warps 5-8 are the epilogue.  Two
// accumulators let a tile's epilogue overlap the next tile's main loop.  Every
// wait is bounded: on expiry the kernel records kStatusTimeout and winds down.
//
// Bound by the tensor cores, and over a long call by the power limit: a stage's
// 128 KB a pair take an SM's 64 bytes a clock from L2 as long (1024 cycles) as
// its MMAs take, so neither a taller nor a wider tile is to be had from this
// much shared memory.  34,502 rows of 7168 x 2048 (gated): 1172 us, 1730
// TFLOP/s, the tensor pipe active 82 % of the cycles; both gradients of 16,407
// rows of 1024 x 4096: 180 us, 1530 TFLOP/s (single launches after a pause; in a
// loop, at the power limit, they take 4 to 8 % longer).  Short contractions over uneven
// rows are bound by the outputs' stores and the last wave: 32 experts x 156
// rows of 1032 x 328, 30 us forward and 51 backward, against 4 and 7 us of
// tensor time.
#include "activation.cuh"
#include "ffn.h"
#include "pair.cuh"
#include "pdl.cuh"
#include "segments.cuh"

namespace a2av {

namespace {

constexpr int BM = 128;        // rows a CTA stages
constexpr int TILE_M = 256;    // rows of a pair's tile
constexpr int BK = 128;        // contraction elements a stage
constexpr uint32_t kAtomBytes = 128 * 128;     // 128 rows x 64 elements
constexpr uint32_t kTileBytes = 2 * kAtomBytes;   // A
constexpr int kMaxStages = 4;
constexpr int kClearWarp = 1;
constexpr int kMmaWarp = 4;
constexpr int kThreads = 9 * 32;

// BN: accumulator columns of a tile, half of them from each CTA's B.
template <int BN>
struct Shape {
    static constexpr int kBRows = BN / 2;  // columns of B a CTA stages
    static constexpr uint32_t kBBytes = kBRows * 256;
    static constexpr uint32_t kStageBytes = kTileBytes + kBBytes;
    static constexpr int kStages = BN == 256 ? 3 : 4;
    static constexpr uint32_t kTmemCols = 2 * BN;
    static constexpr uint32_t kMnAtoms = kBRows / 64;       // B MN-major: atoms of 64 columns
    static constexpr uint32_t kKmAtomBytes = kBRows * 128;  // B K-major: an atom of 64 k
};

struct GroupInfo {
    int32_t row0;   // first expert-major row
    int32_t rows;
    int32_t tile0;  // first tile over its rows
};

struct Control {
    uint64_t full[kMaxStages];    // even CTA: a stage has landed in both CTAs
    uint64_t empty[kMaxStages];   // the MMAs that read a stage have completed
    uint64_t ragged[kMaxStages];  // this CTA's part of a ragged block has landed
    uint64_t cleared[kMaxStages]; // even CTA: both CTAs have cleared a ragged block's rows
    uint64_t tfull[2];         // accumulator ready for the epilogue
    uint64_t tempty[2];        // even CTA: both epilogues have drained it
    uint32_t tmem_base;
    int32_t abort;
    int32_t row_tiles, total_tiles;
    GroupInfo g[kMaxExperts + 1];
    SegmentTable seg;
};

constexpr size_t kControlBytes = (sizeof(Control) + 1023) / 1024 * 1024;
template <int BN>
constexpr size_t smem_bytes() {
    return 1024 + Shape<BN>::kStages * Shape<BN>::kStageBytes + kControlBytes;
}
static_assert(smem_bytes<256>() <= 232448 && smem_bytes<128>() <= 232448, "shared memory per CTA");

struct Tile {
    int g, m, n;
    bool weights;  // of the weights' gradient
    int slice;     // of its contraction
};

// What a launch's tiles cover.
struct Walk {
    int tn;       // column tiles of a tile over rows
    int wm, wn;   // row and column tiles of an expert's weights' gradient
    int slices, w_slices;
};

// The tiles over the experts' rows, then those of the weights' gradients; of
// each expert the row tiles in order, slices in them, column tiles innermost.
__device__ __forceinline__ Tile tile_at(const Control &c, int t, const Walk &k) {
    if (t >= c.row_tiles) {
        const int u = t - c.row_tiles, per = k.wm * k.w_slices * k.wn, local = u % per;
        const int m = local / k.wn;
        return {u / per, m / k.w_slices, local % k.wn, true, m % k.w_slices};
    }
    int g = 0;
    while (t >= c.g[g + 1].tile0) ++g;
    const int local = t - c.g[g].tile0, m = local / k.tn;
    return {g, m / k.slices, local % k.tn, false, m % k.slices};
}

__device__ __forceinline__ void st_global_b32x4(void *ptr, const uint32_t *r) {
    asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(ptr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// 32 bytes, a whole sector, to a 32-byte aligned address.
__device__ __forceinline__ void st_global_b32x8(void *ptr, const uint32_t *r) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Instruction descriptor for kind::f16 with an fp32 accumulator and the
// operands' majors, M = 256.
template <bool BF16, int BN>
__device__ __forceinline__ constexpr uint32_t instr_desc(bool a_mn, bool b_mn) {
    return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(BN >> 3) << 17) | ((256u >> 4) << 24);
}

// Contraction block kb of a tile: its first element and how many of its 128
// elements count.  The weights' gradient takes the ragged last block first.
struct Block {
    int first, len;
};
__device__ __forceinline__ Block block_of(bool weights, int K, int kb) {
    if (weights && K % BK != 0) {
        if (kb == 0) return {K / BK * BK, K % BK};
        return {(kb - 1) * BK, BK};
    }
    return {kb * BK, min(BK, K - kb * BK)};
}

// Contraction blocks of one slice of a tile: those from `first` on, of K's.
struct Span {
    int first, count;
};
__device__ __forceinline__ Span span_of(int K, int slice, int slices) {
    const int blocks = blocks_of(K, BK);
    if (slices == 1) return {0, blocks};
    const int first = static_cast<int>(static_cast<int64_t>(blocks) * slice / slices);
    return {first, static_cast<int>(static_cast<int64_t>(blocks) * (slice + 1) / slices) - first};
}

// Until the count of finished pieces reaches `want`, by one thread; then the
// rows may be read by TMA.  False: gave up.
__device__ __noinline__ bool wait_pieces(int32_t *abort_flag, const int32_t *count, int32_t want, int32_t *status,
                                         uint64_t limit_ns) {
    const auto done = [&]() {
        int32_t v;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
        return v >= want;
    };
    if (!done()) {
        const uint64_t t0 = global_timer_ns();
        while (!done()) {
            __nanosleep(100);
            if (*reinterpret_cast<volatile int32_t *>(abort_flag)) return false;
            if (global_timer_ns() - t0 > limit_ns) {
                *reinterpret_cast<volatile int32_t *>(abort_flag) = 1;
                atomicOr(status, kStatusTimeout);
                return false;
            }
        }
    }
    asm volatile("fence.proxy.async.global;" ::: "memory");
    return true;
}

// GRAD: the gradients' tiles (both kinds); otherwise the gated block's.
template <bool BF16, bool GRAD, int ACT, int BN>
__global__ void __launch_bounds__(kThreads, 1) expert_gemm_kernel(const __grid_constant__ ExpertGemmLaunch p) {
    using S = Shape<BN>;
    constexpr int kStages = S::kStages;
    constexpr uint32_t kStageBytes = S::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    Control &C = *reinterpret_cast<Control *>(base_ptr + kStages * kStageBytes);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = pair::cluster_rank();
    const int unit = blockIdx.x / 2, nunits = gridDim.x / 2;
    // Columns of the output one tile covers; the tiles of a launch.
    const int row_n = GRAD ? BN : BN / 2, w_n = p.half_step ? BN : BN / 2;
    const Walk walk{(p.N + row_n - 1) / row_n, (p.wM + TILE_M - 1) / TILE_M, (p.wN + w_n - 1) / w_n,
                    GRAD ? p.slices : 1, GRAD ? p.w_slices : 1};

    // ---- prologue: groups and tiles (warp 0), barriers (warp 1), TMEM (MMA warp)
    if (warp == 0) {
        // (A kernel that this one overlaps has waited for all before it, and
        // recvCounts was there for it too.)
        const bool overlaps = p.pieces || p.after_permute;
        if (!overlaps) pdl_wait();
        const bool good = build_segments(p.recvCounts, p.W, p.e, p.A, C.seg, lane);
        int row0 = 0, rows = 0, tiles = 0;
        if (lane < p.e) {
            row0 = C.seg.dst[lane * p.W];
            rows = C.seg.dst[(lane + 1) * p.W] - row0;
            tiles = good ? blocks_of(rows, TILE_M) * walk.slices * walk.tn : 0;
        }
        int inc = tiles;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane < p.e) C.g[lane] = GroupInfo{row0, rows, inc - tiles};
        const int total = __shfl_sync(0xffffffffu, inc, 31);
        if (lane == 0) {
            C.g[p.e] = GroupInfo{0, 0, total};
            C.row_tiles = total;
            C.total_tiles = total + (good ? p.e * walk.wm * walk.w_slices * walk.wn : 0);
            C.abort = 0;
            if (blockIdx.x == 0) {
                if (p.write_status) *p.status = good ? 0 : kStatusBadCounts;
                else if (!good) atomicOr(p.status, kStatusBadCounts);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(smem_u32(&C.full[s]), 1);
                mbar_init(smem_u32(&C.empty[s]), 1);
                mbar_init(smem_u32(&C.ragged[s]), 1);
                mbar_init(smem_u32(&C.cleared[s]), 2);
            }
            for (int a = 0; a < 2; ++a) {
                mbar_init(smem_u32(&C.tfull[a]), 1);
                mbar_init(smem_u32(&C.tempty[a]), 8);
            }
            fence_barrier_init();
        }
    } else if (warp == 2) {
        if (lane == 0) {
            if (p.A > 0) {  // (the maps of tiles that there are none of were not made)
                prefetch_tensormap(&p.tmA[0]);
                if (walk.tn > 0) prefetch_tensormap(&p.tmB[GRAD ? 0 : rank]);
                if (walk.wm > 0) prefetch_tensormap(&p.tmX);
            }
        }
    } else if (warp == kMmaWarp) {
        pair::tmem_alloc_pair(smem_u32(&C.tmem_base), S::kTmemCols);
    }
    tc_fence_before_sync();
    pair::sync_all();
    tc_fence_after_sync();

    const int total = C.total_tiles;
    const uint32_t full0 = smem_u32(&C.full[0]), empty0 = smem_u32(&C.empty[0]);
    const uint32_t ragged0 = smem_u32(&C.ragged[0]), cleared0 = smem_u32(&C.cleared[0]);
    const auto contraction = [&](const Tile &w) { return w.weights ? C.g[w.g].rows : p.K; };
    const auto is_ragged = [&](const Tile &w, const Block &b) { return w.weights && (b.len & 15) != 0; };
    const auto span = [&](const Tile &w, int K) { return span_of(K, w.slice, w.weights ? walk.w_slices : walk.slices); };
    // Contraction blocks of a tile: each product's, and those of the second summands.
    const auto steps_of = [&](const Tile &w, int kblocks) {
        return GRAD ? (w.weights ? p.parts : p.phases * p.parts) * kblocks : kblocks;
    };

    if (warp == 0) {
        // =========================================================== producer
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            bool all_there = !p.pieces && !p.after_permute;  // the kernel before this one has completed
            for (int t = unit; t < total && ok; t += nunits) {
                const Tile w = tile_at(C, t, walk);
                const int K = contraction(w);
                const Span ks = span(w, K);
                const int kblocks = ks.count, steps = steps_of(w, kblocks);
                const int g_end = C.g[w.g].row0 + C.g[w.g].rows;
                // This CTA's first row; without a row of its own, any one (nothing of it is stored).
                const int from = w.m * TILE_M + static_cast<int>(rank) * BM;
                const bool live = from < C.g[w.g].rows;
                const int row = C.g[w.g].row0 + (live ? from : 0);
                const CUtensorMap *ta = &p.tmA[0];
                int arow = row;
                if (!GRAD && p.direct_halves && live && half_in_one_segment(C.seg, p.W, p.e, row, g_end)) {
                    // A half whose rows of this group lie in one (source, expert)
                    // run is read where it arrived.
                    ta = &p.tmDirect;
                    arow = source_row(C.seg, p.W, p.e, row);
                } else if (!all_there) {
                    if (!GRAD || w.weights) {  // staged rows, or all rows contracted
                        pdl_wait();
                        all_there = true;
                    } else if (live) {
                        for (int c = row / BM; c <= (run_end(row, BM, g_end) - 1) / BM && ok; ++c)
                            ok = wait_pieces(&C.abort, p.pieces + c, c == p.A / BM ? p.last_pieces : p.row_pieces, p.status,
                                             p.wait_limit_ns);
                        if (!ok) break;
                    }
                }
                for (int i = 0, kb = 0, phase = 0; i < steps; ++i, ++it, ++kb) {
                    const int s = it % kStages;
                    if (kb == kblocks) kb = 0, ++phase;
                    const Block b = block_of(w.weights, K, ks.first + kb);
                    if (!pair::wait_phase(&C.abort, empty0 + 8 * s, ((it / kStages) & 1) ^ 1, p.status,
                                          p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a_st = base + s * kStageBytes, b_st = a_st + kTileBytes;
                    // Where the loads complete: the even CTA's barrier for
                    // both CTAs' parts; a ragged block on each CTA's own.
                    uint32_t bar;
                    if (is_ragged(w, b)) {
                        bar = ragged0 + 8 * s;
                        mbar_arrive_expect_tx(bar, kStageBytes);
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * kStageBytes);
                        bar = pair::map_to_rank(full0 + 8 * s, 0);
                    }
                    int ax, ay, bx, by, bz = w.g;
                    const CUtensorMap *a_map, *b_map;
                    bool one_a = p.one_a, one_b = p.one_b;
                    if constexpr (!GRAD) {
                        a_map = ta, ax = b.first, ay = arow;
                        b_map = &p.tmB[rank], bx = w.n * (BN / 2), by = b.first;
                    } else if (!w.weights) {
                        a_map = &p.tmA[phase], ax = b.first, ay = row;
                        b_map = &p.tmB[phase % p.phases], bx = b.first, by = w.n * BN + static_cast<int>(rank) * S::kBRows;
                    } else {
                        ay = by = C.g[w.g].row0 + b.first;
                        a_map = &p.tmX, ax = w.m * TILE_M + static_cast<int>(rank) * BM;
                        b_map = &p.tmD[phase * p.phases + (p.half_step ? 0 : rank)], bx = w.n * w_n + static_cast<int>(rank) * p.half_step;
                        bz = 0;
                        one_a = p.one_x, one_b = p.one_a;
                    }
                    if (one_a) {
                        pair::load_4d(a_st, a_map, bar, 0, ay, ax / 64, 0);
                    } else {
                        pair::load_3d(a_st, a_map, bar, ax, ay, 0);
                        pair::load_3d(a_st + kAtomBytes, a_map, bar, ax + 64, ay, 0);
                    }
                    if (one_b) {
                        pair::load_4d(b_st, b_map, bar, 0, by, bx / 64, bz);
                    } else {  // the second atom: 64 more columns, or 64 more of K
                        const bool km = GRAD && !w.weights;
                        pair::load_3d(b_st, b_map, bar, bx, by, bz);
                        if (km || S::kMnAtoms == 2)
                            pair::load_3d(b_st + (km ? S::kKmAtomBytes : kAtomBytes), b_map, bar, bx + 64, by, bz);
                    }
                }
            }
            pdl_trigger();
            if (!all_there) pdl_wait();  // (a kernel's end implies that of all before it)
            // Tail: every stage filled has been released (no copy in flight).
            for (int i = 0; i < kStages && ok; ++i, ++it)
                ok = pair::wait_phase(&C.abort, empty0 + 8 * (it % kStages), ((it / kStages) & 1) ^ 1, p.status,
                                      p.wait_limit_ns);
            if (!ok) pair::let_settle();
        }
    } else if (warp == kClearWarp && GRAD) {
        // ============================================= ragged rows of the block
        uint32_t it = 0;
        uint32_t used = 0;  // parity, by stage, of the ragged blocks seen
        bool ok = true;
        for (int t = unit; t < total && ok; t += nunits) {
            const Tile w = tile_at(C, t, walk);
            const int K = contraction(w);
            const Span ks = span(w, K);
            const int kblocks = ks.count;
            const Block b = kblocks ? block_of(w.weights, K, ks.first) : Block{0, 0};
            for (int part = 0; part < (is_ragged(w, b) ? p.parts : 0) && ok; ++part) {
                const int s = (it + part * kblocks) % kStages;
                ok = pair::wait_phase_warp(&C.abort, ragged0 + 8 * s, (used >> s) & 1, p.status, p.wait_limit_ns);
                if (!ok) break;
                used ^= 1u << s;
                // Rows len .. the next multiple of 16, 128 bytes in each atom of
                // A and B (the swizzle stays within a row): eight lanes an atom.
                const uint32_t st = base + s * kStageBytes + b.len * 128 + (lane / 8) * kAtomBytes + (lane % 8) * 16;
                if (lane / 8 < 2 + S::kMnAtoms)
                    for (int r = b.len & 15; r < 16; ++r) st_shared_v4(st + (r - (b.len & 15)) * 128, make_uint4(0, 0, 0, 0));
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    pair::arrive_cluster(pair::map_to_rank(cleared0 + 8 * s, 0));
                    if (rank == 0) mbar_arrive(full0 + 8 * s);  // the stage's phase, in place of the loads' bytes
                }
            }
            it += steps_of(w, kblocks);
        }
    } else if (warp == kMmaWarp) {
        // =========================================================== MMA issuer
        if (lane == 0 && rank == 0) {
            // K-major: 8-row groups 1024 B apart; a K step of 16 elements is
            //    32 B along the row, the second atom 16 KB on.
            // MN-major: atoms of 64 columns 16 KB apart (leading offset), 8-row
            //    K groups 1024 B apart; a K step of 16 rows is 2 KB.
            const uint64_t desc_km = smem_desc(base, 16, 1024, kSwizzle128B);
            const uint64_t desc_mn = smem_desc(base, kAtomBytes, 1024, kSwizzle128B);
            const uint64_t to_b = kTileBytes >> 4;
            uint32_t it = 0, tl = 0, used = 0;
            bool ok = true;
            for (int t = unit; t < total && ok; t += nunits, ++tl) {
                const Tile w = tile_at(C, t, walk);
                const int K = contraction(w);
                const Span ks = span(w, K);
                const int kblocks = ks.count, steps = steps_of(w, kblocks);
                const int acc = tl & 1;
                // A: MN-major for the weights' gradient only; B: K-major for the rows' gradient only.
                const bool a_is_mn = GRAD && w.weights, b_is_mn = !GRAD || w.weights;
                const uint32_t idesc = instr_desc<BF16, BN>(a_is_mn, b_is_mn);
                const uint64_t a_desc0 = a_is_mn ? desc_mn : desc_km;
                const uint64_t b_desc0 = (b_is_mn ? desc_mn : desc_km) + to_b;
                if (!pair::wait_phase(&C.abort, smem_u32(&C.tempty[acc]), ((tl >> 1) & 1) ^ 1, p.status,
                                      p.wait_limit_ns))
                    break;
                tc_fence_after_sync();
                const uint32_t d_tmem = C.tmem_base + acc * BN;
                for (int i = 0, kb = 0; i < steps; ++i, ++it, ++kb) {
                    const int s = it % kStages;
                    if (kb == kblocks) kb = 0;
                    const uint32_t par = (it / kStages) & 1;
                    if (!mbar_try_wait(full0 + 8 * s, par) &&
                        !pair::wait_phase(&C.abort, full0 + 8 * s, par, p.status, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const Block b = block_of(w.weights, K, ks.first + kb);
                    if (is_ragged(w, b)) {
                        if (!pair::wait_phase(&C.abort, cleared0 + 8 * s, (used >> s) & 1, p.status,
                                              p.wait_limit_ns)) {
                            ok = false;
                            break;
                        }
                        used ^= 1u << s;
                        tc_fence_after_sync();
                    }
                    const uint64_t ad0 = a_desc0 + ((s * kStageBytes) >> 4);
                    const uint64_t bd0 = b_desc0 + ((s * kStageBytes) >> 4);
                    const int ksteps = (b.len + 15) / 16;
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        if (kk < ksteps) {
                            const uint32_t mn = 128 * kk;
                            const uint32_t a_km = ((kk >> 2) * kAtomBytes + (kk & 3) * 32) >> 4;
                            const uint32_t b_km = ((kk >> 2) * S::kKmAtomBytes + (kk & 3) * 32) >> 4;
                            pair::mma(d_tmem, ad0 + (a_is_mn ? mn : a_km), bd0 + (b_is_mn ? mn : b_km), idesc,
                                      (i | kk) != 0);
                        }
                    }
                    pair::commit(empty0 + 8 * s);
                }
                if (ok) pair::commit(smem_u32(&C.tfull[acc]));
            }
        }
    } else if (warp > kMmaWarp) {
        // =========================================================== epilogue
        const int q = warp & 3;  // TMEM lane quarter this warp may read
        const uint32_t tempty0 = pair::map_to_rank(smem_u32(&C.tempty[0]), 0);
        uint32_t tl = 0;
        for (int t = unit; t < total; t += nunits, ++tl) {
            const Tile w = tile_at(C, t, walk);
            const int acc = tl & 1;
            if (!pair::wait_phase_warp(&C.abort, smem_u32(&C.tfull[acc]), (tl >> 1) & 1, p.status, p.wait_limit_ns)) break;
            tc_fence_after_sync();
            const GroupInfo gi = C.g[w.g];
            const int row0w = w.m * TILE_M + static_cast<int>(rank) * BM + q * 32;  // this warp's first row
            const int rows = w.weights ? p.wM : gi.rows, N = w.weights ? p.wN : p.N;
            const bool valid = row0w + lane < rows;
            // Output row of this lane's row.
            int64_t orow = 0;
            if (w.weights) {
                orow = static_cast<int64_t>(w.g) * p.wM + row0w + lane;
            } else if constexpr (!GRAD) {
                orow = static_cast<int64_t>(gi.row0) + row0w + lane;
            } else if (valid) {  // the gradient's rows go back to their order of arrival
                orow = source_row(C.seg, p.W, p.e, gi.row0 + row0w + lane);
            }
            const bool zero = GRAD && span(w, contraction(w)).count == 0;  // nothing was accumulated
            const int slices = w.weights ? walk.w_slices : walk.slices;
            const uint32_t t_base = C.tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
            const bool wide = N % 16 == 0;
            constexpr int kChunks = GRAD ? BN / 32 : BN / 64;
            for (int c = 0; c < kChunks; ++c) {
                const int half = c / (BN / 64);
                const int col = !GRAD ? w.n * (BN / 2) + c * 32
                                      : !w.weights ? w.n * BN + c * 32
                                                   : w.n * w_n + half * p.half_step + c % (BN / 64) * 32;
                if (col >= N) continue;  // uniform
                uint32_t r[32];
                tmem_ld_32x32b_x32(t_base + c * 32, r);
                if constexpr (!GRAD) {
                    uint32_t u[32];
                    tmem_ld_32x32b_x32(t_base + BN / 2 + c * 32, u);
                    tmem_ld_wait();
                    if (p.saved[0] && valid) {
                        float *g_out = p.saved[0] + orow * p.N + col, *u_out = p.saved[1] + orow * p.N + col;
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            if (col + v * 8 < p.N) {
                                st_global_b32x8(g_out + v * 8, r + v * 8);
                                st_global_b32x8(u_out + v * 8, u + v * 8);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float a, b;
                        split(mul2(act_value<ACT>(pair_of(__uint_as_float(r[i]), __uint_as_float(r[i + 1]))),
                                   pair_of(__uint_as_float(u[i]), __uint_as_float(u[i + 1]))),
                              a, b);
                        r[i] = __float_as_uint(a);
                        r[i + 1] = __float_as_uint(b);
                    }
                } else {
                    tmem_ld_wait();
                    if (zero) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = 0;
                    }
                    if (slices > 1) {
                        if (valid) {
                            const int64_t m = w.weights ? (p.half_step ? 0 : half) * slices + w.slice : w.slice;
                            float *const to = (w.weights ? p.part_w : p.part) +
                                              (m * (w.weights ? static_cast<int64_t>(p.e) * p.wM : p.A) + orow) * N + col;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                if (col + v * 8 < N) st_global_b32x8(to + v * 8, r + v * 8);
                        }
                        continue;
                    }
                }
                uint32_t w16[16];
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    w16[v] = pack2<BF16>(pair_of(__uint_as_float(r[2 * v]), __uint_as_float(r[2 * v + 1])));
                if (valid) {
                    uint16_t *const out = static_cast<uint16_t *>(w.weights ? p.out_w[half] : p.out) + orow * N + col;
                    if (wide && (reinterpret_cast<uintptr_t>(out) & 31) == 0) {
#pragma unroll
                        for (int v = 0; v < 2; ++v)
                            if (col + v * 16 < N) st_global_b32x8(out + v * 16, w16 + v * 8);
                    } else {
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (col + v * 8 < N) st_global_b32x4(out + v * 8, w16 + v * 4);
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) pair::arrive_reads_done(tempty0 + 8 * acc);
        }
    }

    __syncwarp();  // the single-lane roles are done
    tc_fence_before_sync();
    pair::sync_all();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        pair::tmem_free_pair(C.tmem_base, S::kTmemCols);
    }
}

// The gradients' slices joined: out = the sum over slices of part, in order, for
// up to three matrices, eight values a thread.  Bound by the sums' bytes, which
// are in L2 where there are few: 4 slices of 448 x 896, 3 us behind the GEMM.
struct Join {
    const float *part[3];
    void *out[3];
    int64_t vecs[3];  // of a slice
    int32_t slices[3];
    const int32_t *status;
};
constexpr int kJoinThreads = 128;
template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Join p) {
    pdl_trigger();
    pdl_wait();
    if (*p.status != 0) return;  // the slices were not all written
    int64_t v = static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x;
    int i = 0;
    while (i < 3 && v >= p.vecs[i]) v -= p.vecs[i++];
    if (i == 3) return;
    const float4 *from = reinterpret_cast<const float4 *>(p.part[i]) + 2 * v;
    float4 lo = __ldcs(from), hi = __ldcs(from + 1);
#pragma unroll 4
    for (int s = 1; s < p.slices[i]; ++s) {
        from += 2 * p.vecs[i];
        const float4 a = __ldcs(from), b = __ldcs(from + 1);
        lo = make_float4(lo.x + a.x, lo.y + a.y, lo.z + a.z, lo.w + a.w);
        hi = make_float4(hi.x + b.x, hi.y + b.y, hi.z + b.z, hi.w + b.w);
    }
    const f32x2 o[4] = {pair_of(lo.x, lo.y), pair_of(lo.z, lo.w), pair_of(hi.x, hi.y), pair_of(hi.z, hi.w)};
    static_cast<uint4 *>(p.out[i])[v] = pack8<BF16>(o);
}

cudaError_t launch_join(const ExpertGemmLaunch &p, cudaStream_t stream) {
    Join j = {};
    int64_t total = 0;
    const auto add = [&](int i, const float *part, void *out, int64_t values, int slices) {
        j.part[i] = part;
        j.out[i] = out;
        j.vecs[i] = values / 8;
        j.slices[i] = slices;
        total += j.vecs[i];
    };
    if (p.N > 0 && p.slices > 1) add(0, p.part, p.out, static_cast<int64_t>(p.A) * p.N, p.slices);
    const int64_t matrix = static_cast<int64_t>(p.e) * p.wM * p.wN;
    for (int i = 0; p.wM > 0 && p.w_slices > 1 && i < (p.half_step ? 1 : 2); ++i)
        add(1 + i, p.part_w + i * p.w_slices * matrix, p.out_w[i], matrix, p.w_slices);
    if (total == 0) return cudaSuccess;
    j.status = p.status;
    const unsigned blocks = static_cast<unsigned>((total + kJoinThreads - 1) / kJoinThreads);
    return p.bf16 ? launch_pdl(join_kernel<true>, blocks, kJoinThreads, 0, 0, stream, j)
                  : launch_pdl(join_kernel<false>, blocks, kJoinThreads, 0, 0, stream, j);
}

template <bool BF16, bool GRAD, int ACT, int BN>
cudaError_t launch_shape(const ExpertGemmLaunch &p, cudaStream_t stream) {
    auto kern = expert_gemm_kernel<BF16, GRAD, ACT, BN>;
    const cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_bytes<BN>()));
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, p.grid, kThreads, smem_bytes<BN>(), 2, stream, p);
}

template <bool BF16, bool GRAD, int ACT>
cudaError_t launch_kind(const ExpertGemmLaunch &p, cudaStream_t stream) {
    return p.bn == 256 ? launch_shape<BF16, GRAD, ACT, 256>(p, stream) : launch_shape<BF16, GRAD, ACT, 128>(p, stream);
}

template <bool BF16>
cudaError_t launch_type(const ExpertGemmLaunch &p, cudaStream_t stream) {
    if (p.grad) return launch_kind<BF16, true, A2AV_ACT_SILU>(p, stream);
    return p.act == A2AV_ACT_SILU ? launch_kind<BF16, false, A2AV_ACT_SILU>(p, stream)
                                  : launch_kind<BF16, false, A2AV_ACT_GELU_TANH>(p, stream);
}

}  // namespace

cudaError_t launch_expert_gemm(const ExpertGemmLaunch &p, cudaStream_t stream) {
    const cudaError_t err = p.bf16 ? launch_type<true>(p, stream) : launch_type<false>(p, stream);
    return err == cudaSuccess && p.grad ? launch_join(p, stream) : err;
}

// Every kind needs nearly all of an SM's shared memory: one CTA an SM.
int expert_gemm_max_clusters() {
    return max_clusters(expert_gemm_kernel<true, false, A2AV_ACT_SILU, 256>, kThreads, smem_bytes<256>(), 2);
}

}  // namespace a2av
