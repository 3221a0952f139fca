// The product of 8-bit rows with a float32 scale per 128 codes for few rows an
// expert (decode and small batches):
//
//   y[i][n] = sum over b of xs[i][b] ws[n / 128][b] sum over k in b of x[i][k] w[n][k]
//
// Bound by the bytes of the weights of the experts that have rows, so the weights
// stream: 128 of their columns are the M operand of tcgen05.mma, up to 16 rows of x
// the narrow one (N), both K-major as they lie in memory.  A stage is a
// K block of 128 codes, which has one scale a row and one for its columns: four
// MMAs into a TMEM accumulator of its own, which the epilogue scales and adds to
// sums in registers (a lane has a column of the weights, a register a row of x).
//
// A job is (unit of up to 16 rows of an expert, 128 columns).  How many there are
// is known on the device only, so the K blocks of all jobs, one behind the other,
// are cut into one equal piece a CTA.  A job that several CTAs share has its sums
// put into the workspace by each; the last of them to come adds all in order: the
// same result every time, whoever it is.
//
// A kernel before it puts the rows' scales in expert-major order, a K block's next
// to each other, and the rows themselves where they come from several sources.
// Per CTA: warp 0 loads the weights, from before that kernel's end; warp 2 the rows;
// warp 1 issues the MMAs; warps 4-11 are the epilogue, two for each TMEM lane
// quarter, half of the rows each.  Every wait is bounded.
//
// 8 rows over 4 experts of 4096 x 2048 (34 MB of weights where all have rows): 14 to
// 15 us a call; a kernel that does nothing but read as much from HBM takes 12.5.
#include <algorithm>

#include "activation.cuh"
#include "g128.h"
#include "pair.cuh"
#include "pdl.cuh"
#include "segments.cuh"

namespace a2av {

namespace {

constexpr int kMmaWarp = 1;
constexpr int kRowWarp = 2;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr int kBK = 128;                  // codes of a K block
constexpr int kCols = 128;                // columns of a job
constexpr uint32_t kWBytes = kCols * kBK;
constexpr int R = kG128UnitRows;
static_assert(R == 16, "the sizes below are made for it");
constexpr uint32_t kStage = kWBytes + R * kBK;
constexpr int kStages = 12;
constexpr int kAccs = 4;                  // accumulators
constexpr uint32_t kTmemCols = kAccs * R;
constexpr int kOwn = R / 2;               // rows of an epilogue warp

struct Control {
    uint64_t full[kStages], empty[kStages];
    uint64_t tfull[kAccs], tempty[kAccs];
    uint32_t tmem_base;
    int32_t abort;
    int32_t arrived;                    // what this CTA's arrival at a shared job found
    int32_t units;
    int32_t start[kMaxExperts + 1];     // first unit of each expert
    alignas(16) float scale[kEpiWarps][kOwn];  // of a warp's rows
    SegmentTable seg;
};
constexpr size_t kControlBytes = (sizeof(Control) + 1023) / 1024 * 1024;

constexpr size_t kSmem = 1024 + kStages * kStage + kControlBytes;
static_assert(kSmem <= 232448, "shared memory per CTA");

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 8 consecutive columns, and the wait behind which they are used.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld8_wait(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// All threads of the epilogue; the second, and whether all of them say yes: a
// warp whose wait was given up takes the others along.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory"); }
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

// A ring's place: stage (or accumulator) and how often it has been gone round.
struct Place {
    int s = 0, turn = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) s = 0, ++turn;
    }
};

// Rows [first, first + rows) of expert-major order, and their expert.
struct Unit {
    int expert, first, rows;
};

// Scales (and rows) in expert-major order; clears the status and the arrivals.  A
// warp a row.
constexpr int kStageWarps = 8;
__global__ void __launch_bounds__(kStageWarps * 32) g128_stage_kernel(const __grid_constant__ G128Stage p) {
    __shared__ SegmentTable table;
    __shared__ int ok;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_wait();
    if (blockIdx.x == 0) {  // before the kernel behind this one can set bits of the status
        if (threadIdx.x == 0) *p.status = 0;
        for (int i = threadIdx.x; i < kG128Ctas; i += kStageWarps * 32) p.arrivals[i] = 0;
        __threadfence();
        __syncthreads();
    }
    pdl_trigger();
    if (warp == 0) {
        const bool good = build_segments(p.recvCounts, p.W, p.e, p.A, table, lane);
        if (lane == 0) ok = good;
    }
    __syncthreads();
    if (!ok) return;  // (the kernel behind this one reports it)
    const int kblocks = p.K / kBK, vecs = p.K / 16;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kStageWarps + warp; row < p.A;
         row += static_cast<int64_t>(gridDim.x) * kStageWarps) {
        const int64_t from = source_row(table, p.W, p.e, static_cast<int32_t>(row));
        if (p.dst) {
            const uint4 *in = static_cast<const uint4 *>(p.src) + from * vecs;
            uint4 *out = static_cast<uint4 *>(p.dst) + row * vecs;
#pragma unroll 4
            for (int v = lane; v < vecs; v += 32) out[v] = in[v];
        }
        for (int b = lane; b < kblocks; b += 32) p.scales[static_cast<int64_t>(b) * p.A + row] = p.xs[from * kblocks + b];
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) g128_rows_kernel(const __grid_constant__ G128Launch p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    Control &C = *reinterpret_cast<Control *>(smem_raw + (base - raw) + kStages * kStage);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int strips = (p.N + kCols - 1) / kCols, kblocks = p.K / kBK;

    if (warp == 0) {
        // (The kernel before this one, which stages the rows and has cleared the status
        // and the arrivals, let it start after all before that one had completed.)
        const bool good = build_segments(p.recvCounts, p.W, p.e, p.A, C.seg, lane);
        int units = 0;
        if (lane < p.e && good) units = blocks_of(C.seg.dst[(lane + 1) * p.W] - C.seg.dst[lane * p.W], R);
        int inc = units;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane < p.e) C.start[lane] = inc - units;
        if (lane == 31) {
            C.start[p.e] = inc;
            C.units = inc;
            C.abort = 0;
            if (blockIdx.x == 0 && !good) atomicOr(p.status, kStatusBadCounts);
        }
    } else if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&C.tmem_base), kTmemCols);
        tmem_relinquish();
    } else if (warp == kEpiWarp0) {
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(smem_u32(&C.full[s]), 2);
                mbar_init(smem_u32(&C.empty[s]), 1);
            }
            for (int a = 0; a < kAccs; ++a) {
                mbar_init(smem_u32(&C.tfull[a]), 1);
                mbar_init(smem_u32(&C.tempty[a]), kEpiWarps);
            }
            fence_barrier_init();
        }
    } else if (warp == kEpiWarp0 + 1 && lane == 0) {
        prefetch_tensormap(&p.tmA);
        prefetch_tensormap(&p.tmB);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();

    // The K blocks of all jobs, and this CTA's (each has one at least: a job's shares
    // are those of consecutive CTAs).
    const int units = __shfl_sync(0xffffffffu, C.units, 0);
    const int64_t total = static_cast<int64_t>(units) * strips * kblocks;
    const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total)), me = blockIdx.x;
    const auto begin_of = [&](int cta) { return total * cta / ctas; };
    const auto owner_of = [&](int64_t step) { return static_cast<int>(((step + 1) * ctas - 1) / total); };
    const int64_t begin = me < ctas ? begin_of(me) : 0, end = me < ctas ? begin_of(me + 1) : 0;
    const int count = static_cast<int>(end - begin);
    // Of the first K block: its job and its place in it.
    const int64_t job0 = begin / kblocks;
    const int block0 = static_cast<int>(begin % kblocks);
    const int unit0 = static_cast<int>(job0 / strips), strip0 = static_cast<int>(job0 % strips);
    const auto unit_at = [&](int u) {
        int e = 0;
        while (u >= C.start[e + 1]) ++e;
        const int row0 = C.seg.dst[e * p.W], from = (u - C.start[e]) * R;
        return Unit{e, row0 + from, min(R, C.seg.dst[(e + 1) * p.W] - row0 - from)};
    };
    const uint32_t full0 = smem_u32(&C.full[0]), empty0 = smem_u32(&C.empty[0]);
    const uint32_t tfull0 = smem_u32(&C.tfull[0]), tempty0 = smem_u32(&C.tempty[0]);

    if (warp == 0 || warp == kRowWarp) {
        // =========================================================== producers: weights, rows
        // (The whole warp goes along and one lane issues, which leaves the operands in
        // uniform registers.)
        const bool rows = warp == kRowWarp, leader = elect_one();
        const uint32_t bytes = rows ? R * kBK : kWBytes, to = base + (rows ? kWBytes : 0);
        const CUtensorMap *const map = rows ? &p.tmA : &p.tmB;
        // The weights' first stages go out before the kernel that stages the rows has
        // ended.  (The time that a wait may take starts behind it.)
        const int ahead = rows ? 0 : kStages;
        bool ok = true;
        Place at;
        int unit = unit0, strip = strip0, block = block0;
        Unit u = count > 0 ? unit_at(unit) : Unit{0, 0, 0};
        for (int i = 0; i < count; ++i, at.next(kStages)) {
            if (i == ahead) pdl_wait();
            if (at.turn > 0 && !pair::wait_phase_warp(&C.abort, empty0 + 8 * at.s, (at.turn & 1) ^ 1, p.status,
                                                      p.wait_limit_ns)) {
                ok = false;
                break;
            }
            if (leader) {
                mbar_arrive_expect_tx(full0 + 8 * at.s, bytes);
                tma_load_3d(to + at.s * kStage, map, full0 + 8 * at.s, block * kBK, rows ? u.first : strip * kCols,
                            rows ? 0 : u.expert);
            }
            __syncwarp();
            if (++block == kblocks) {
                block = 0;
                if (++strip == strips) {
                    strip = 0;
                    if (i + 1 < count) u = unit_at(++unit);
                }
            }
        }
        if (count <= ahead) pdl_wait();  // (a kernel's end implies that of all before it)
        if (!rows) pdl_trigger();
        // The stages that were filled have been read.
        for (int i = 0; i < kStages && ok; ++i) {
            const int turns = at.s > i ? at.turn + 1 : at.turn;  // fills of stage i
            if (turns > 0)
                ok = pair::wait_phase_warp(&C.abort, empty0 + 8 * i, (turns - 1) & 1, p.status, p.wait_limit_ns);
        }
        if (!ok) pair::let_settle();
    } else if (warp == kMmaWarp) {
        // =========================================================== MMA issuer
        pdl_wait();
        const bool leader = elect_one();
        const uint32_t qtype = static_cast<uint32_t>(p.qtype);
        const uint32_t idesc = (1u << 4) | (qtype << 7) | (qtype << 10) | (static_cast<uint32_t>(R >> 3) << 17) |
                               ((128u >> 4) << 24);
        const uint64_t a_desc0 = smem_desc(base, 16, 1024, kSwizzle128B);
        const uint64_t b_desc0 = smem_desc(base + kWBytes, 16, 1024, kSwizzle128B);
        const uint32_t tmem = __shfl_sync(0xffffffffu, C.tmem_base, 0);
        Place at, acc;
        for (int i = 0; i < count; ++i, at.next(kStages), acc.next(kAccs)) {
            if (!pair::wait_phase_warp(&C.abort, tempty0 + 8 * acc.s, (acc.turn & 1) ^ 1, p.status, p.wait_limit_ns) ||
                !pair::wait_phase_warp(&C.abort, full0 + 8 * at.s, at.turn & 1, p.status, p.wait_limit_ns))
                break;
            tc_fence_after_sync();
            const uint64_t off = static_cast<uint32_t>(at.s * kStage) >> 4;
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < kBK / 32; ++kk)
                    mma_f8(tmem + acc.s * R, a_desc0 + off + 2 * kk, b_desc0 + off + 2 * kk, idesc, kk > 0);
                mma_commit(empty0 + 8 * at.s);
                mma_commit(tfull0 + 8 * acc.s);
            }
            __syncwarp();
        }
    } else if (warp >= kEpiWarp0) {
        // =========================================================== sums and stores
        pdl_wait();
        const int q = warp & 3, half = (warp - kEpiWarp0) / 4, tid = threadIdx.x - kEpiWarp0 * 32;
        const uint32_t t_base = C.tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * kOwn;
        float *const scales = C.scale[warp - kEpiWarp0];
        const size_t slot = static_cast<size_t>(R) * kCols;
        // The sums of a CTA's share of a job: its first (begun by a CTA before it) or its last one.
        const auto share_of = [&](int cta, int owner) { return p.sums + (2 * static_cast<size_t>(cta) + (cta == owner)) * slot; };
        Place acc;
        int unit = unit0, strip = strip0, block = block0;
        Unit u = count > 0 ? unit_at(unit) : Unit{0, 0, 0};
        const float *ws = p.ws, *xs = p.xs;  // scales of the job's columns, and of this warp's rows, of the next K block
        float x = 0.0f, w = 0.0f;
        const auto fetch = [&]() {
            w = *ws;
            x = lane < kOwn && half * kOwn + lane < u.rows ? xs[lane] : 0.0f;
            ++ws;
            xs += p.A;
        };
        const auto prepare = [&]() {
            ws = p.ws + (static_cast<size_t>(u.expert) * strips + strip) * kblocks + block;
            xs = p.xs + static_cast<size_t>(block) * p.A + u.first + half * kOwn;
            fetch();
        };
        if (count > 0) prepare();
        for (int i = 0; i < count;) {
            const int blocks = min(kblocks - block, count - i);  // of this job
            const int col0 = strip * kCols + q * 32, row0 = u.first + half * kOwn, rows = min(kOwn, u.rows - half * kOwn);
            f32x2 sum[kOwn / 2];
#pragma unroll
            for (int j = 0; j < kOwn / 2; ++j) sum[j] = 0;
            bool ok = true;
            for (int b = 0; b < blocks; ++b, acc.next(kAccs)) {
                if (lane < kOwn) scales[lane] = x * w;
                if (b + 1 < blocks) fetch();
                __syncwarp();
                if (!pair::wait_phase_warp(&C.abort, tfull0 + 8 * acc.s, acc.turn & 1, p.status, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                uint32_t r[8];
                tmem_ld8(t_base + acc.s * R, r);
                tmem_ld8_wait(r);
                tc_fence_before_sync();
                if (lane == 0) mbar_arrive(tempty0 + 8 * acc.s);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 s = *reinterpret_cast<const float4 *>(scales + 4 * j);
                    const uint32_t *v = &r[4 * j];
                    sum[2 * j] = fma2(pair_of(__uint_as_float(v[0]), __uint_as_float(v[1])), pair_of(s.x, s.y), sum[2 * j]);
                    sum[2 * j + 1] =
                        fma2(pair_of(__uint_as_float(v[2]), __uint_as_float(v[3])), pair_of(s.z, s.w), sum[2 * j + 1]);
                }
                __syncwarp();  // the scales have been read
            }
            if (!epilogue_all(ok)) break;
            const int64_t first = begin + i - block;  // of the job's K blocks
            const bool whole = blocks == kblocks;
            i += blocks;
            block = 0;
            if (++strip == strips) {
                strip = 0;
                if (i < count) u = unit_at(++unit);
            }
            if (i < count) prepare();  // (its loads are on their way meanwhile)
            // Rows r and r + 1 of this lane's column: two neighbouring columns of one row
            // a lane, 64 bytes of each row a store (N is a multiple of 8).
            const auto store = [&](int r, float a, float b) {
                const bool odd = lane & 1;
                const float other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                const int row = r + odd, col = col0 + (lane & ~1);
                if (row < rows && col < p.N)
                    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.y) + static_cast<size_t>(row0 + row) * p.N + col) =
                        pack2<BF16>(odd ? pair_of(other, b) : pair_of(a, other));
            };
            if (whole) {
#pragma unroll
                for (int j = 0; j < kOwn / 2; ++j) {
                    float a, b;
                    split(sum[j], a, b);
                    if (2 * j < rows) store(2 * j, a, b);
                }
            } else {
                const int owner = owner_of(first), shares = owner_of(first + kblocks - 1) - owner + 1;
                const int at = half * kOwn * kCols + q * 32 + lane;
                float *const share = share_of(me, owner) + at;
#pragma unroll
                for (int j = 0; j < kOwn / 2; ++j) {
                    float a, b;
                    split(sum[j], a, b);
                    if (2 * j < rows) share[2 * j * kCols] = a;
                    if (2 * j + 1 < rows) share[(2 * j + 1) * kCols] = b;
                }
                __threadfence();
                epilogue_sync();
                if (tid == 0) C.arrived = atomicAdd(p.arrivals + owner, 1);
                epilogue_sync();
                if (C.arrived == shares - 1) {
                    __threadfence();
                    // Two shares are asked for together, and added in order.  (The instructions of
                    // more, which every CTA fetches for this once, cost more than they save.)
                    float v[kOwn] = {};
                    for (int k = 0; k < shares; k += 2) {
                        const float *const a = share_of(owner + k, owner) + at;
                        const float *const b = share_of(owner + min(k + 1, shares - 1), owner) + at;
                        float x[kOwn], y[kOwn];
#pragma unroll
                        for (int j = 0; j < kOwn; ++j) {
                            x[j] = j < rows ? __ldcg(a + j * kCols) : 0.0f;
                            y[j] = j < rows && k + 1 < shares ? __ldcg(b + j * kCols) : 0.0f;
                        }
#pragma unroll
                        for (int j = 0; j < kOwn; ++j) v[j] = v[j] + x[j] + y[j];
                    }
#pragma unroll
                    for (int j = 0; j < kOwn; j += 2)
                        if (j < rows) store(j, v[j], v[j + 1]);
                }
                epilogue_sync();  // C.arrived has been read
            }
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(C.tmem_base, kTmemCols);
    }
}

template <bool BF16>
cudaError_t launch_type(const G128Launch &p, cudaStream_t stream) {
    auto kern = g128_rows_kernel<BF16>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, kG128Ctas, kThreads, kSmem, 0, stream, p);
}

}  // namespace

cudaError_t launch_g128_stage(const G128Stage &p, cudaStream_t stream) {
    const int blocks = std::max(1, std::min((p.A + kStageWarps - 1) / kStageWarps, 4 * kG128Ctas));
    return launch_pdl(g128_stage_kernel, blocks, kStageWarps * 32, 0, 0, stream, p);
}

cudaError_t launch_g128_rows(const G128Launch &p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_type<true>(p, stream) : launch_type<false>(p, stream);
}

}  // namespace a2av
