// C ABI of the expert-layer operators (declared in include/a2av_ffn.h):
// argument checks, tensor maps and launches.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "a2av_ffn.h"
#include "ffn.h"
#include "kernels.h"
#include "per_device.h"
#include "plan.cuh"
#include "quantise.cuh"

namespace {

using a2av::ExpertGemmLaunch;

constexpr size_t kStatusBytes = 256;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // bound on every device-side wait
#ifdef A2AV_CHECKS
// Debug builds can make a wait run out: slopes_short holds back one piece of every
// 128 rows' slopes from the GEMM that waits for them.
bool slopes_short = false;
uint64_t wait_limit_ns = kWaitLimitNs;
#else
constexpr uint64_t wait_limit_ns = kWaitLimitNs;
#endif
// Whether the slopes of a backward pass are computed beside its GEMM, which hides
// them but leaves them one block an SM: where that GEMM is long, in each of its
// contractions too.  Measured (us, one after the other / beside; rows x H1 x N of
// a whole training step): 20,000 x 2048 x 1408 526 / 485, 20,000 x 768 x 1408 291
// / 270, 8917 x 2048 x 1408 270 / 258, 2500 x 4096 x 4096 590 / 586; 10,000 x
// 1024 x 1024 141 / 139, 60,000 x 512 x 1024 475 / 488, 30,000 x 4096 x 256 378 /
// 386, 60,000 x 256 x 512 223 / 249.
bool slopes_beside(int64_t A, int64_t H1, int64_t N) {
    return static_cast<double>(A) * H1 * N >= 2e10 && H1 >= 768 && N >= 512;
}
// Mean rows of a (source, expert) run from which whole halves are read in place
// (us, in place / all rows staged; mean run): 5013 rows of 1032 x 328 (20) 35.1
// / 29.2, 20,000 of 2048 x 1408 (78) 175 / 165, 34,502 of 7168 x 2048 (135) 1294
// / 1286, 65,308 of 2048 x 1408 (255) 473 / 482, 16,407 of 4096 x 1024 (513)
// 161 / 188.
constexpr int64_t kLongRun = 96;
// Pairs of SMs, each of which has a tile at a time, of a GB300.  Not asked of the
// device: the workspace's size depends on it, and is asked for without one.
constexpr int64_t kPairs = 76;
bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool mult8(int64_t v) { return v % 8 == 0; }
bool type16(int32_t dtype) { return dtype == A2AV_BF16 || dtype == A2AV_FP16; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

int current_device() {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

int sm_count() {
    static a2av::PerDevice<int> cache;
    const int dev = current_device();
    const int *n = cache.get(dev, [dev](int &v) {
        return cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
    });
    return n ? *n : 0;
}

int gemm_clusters() {
    static a2av::PerDevice<int> cache;
    const int *n = cache.get(current_device(), [](int &v) { return (v = a2av::expert_gemm_max_clusters()) > 0; });
    return n ? *n : 0;
}

// The 8-bit output asked for: its type and mode within the formats, and rows
// that are whole scale blocks.
a2av_status check_quant(int32_t qtype, int32_t qmode, int64_t cols) {
    if (qtype == A2AV_Q_NONE) return A2AV_OK;
    if (qtype < A2AV_Q_E4M3FN || qtype > A2AV_Q_INT8) return A2AV_ERR_INVALID;
    if (qmode != A2AV_QMODE_MX && qmode != A2AV_QMODE_GROUP128) return A2AV_ERR_INVALID;
    if (qmode == A2AV_QMODE_MX && qtype == A2AV_Q_INT8) return A2AV_ERR_INVALID;
    if (cols % (qmode == A2AV_QMODE_MX ? 32 : 128) != 0) return A2AV_ERR_INVALID;
    return A2AV_OK;
}

int kind_of(int32_t qtype, int32_t qmode) {
    return qtype == A2AV_Q_NONE ? a2av::kQuantNone : a2av::quant_kind(qmode, qtype);
}

a2av_status check_quant_out(int32_t qtype, int32_t qmode, const void *codes, const void *scales, bool rows) {
    if (qtype == A2AV_Q_NONE) return codes || scales ? A2AV_ERR_INVALID : A2AV_OK;
    if (rows && (!codes || !scales)) return A2AV_ERR_NULLPTR;
    if (!aligned(codes, 8) || (qmode == A2AV_QMODE_GROUP128 && !aligned(scales, 4))) return A2AV_ERR_UNSUPPORTED;
    return A2AV_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Operand tiles of [groups][rows][cols] row-major: 128 rows x 128 elements (or
// another box) as 64-element atoms, 128-byte swizzled.  `one`: the 4-D view
// [groups][cols / 64][rows][64], all atoms in one box (cols a multiple of 64);
// otherwise the 3-D view, one atom a box.
bool operand_map(CUtensorMap *m, const void *ptr, int64_t groups, int64_t rows, int64_t cols, bool bf16, bool one,
                 uint32_t box_rows = 128, uint32_t atoms = 2) {
    auto fn = encode_fn();
    if (!fn) return false;
    const auto type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t pitch = static_cast<cuuint64_t>(cols) * 2;
    const cuuint64_t plane = groups > 1 ? pitch * rows : pitch;  // not used with one group
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r;
    if (one) {
        const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64),
                                    static_cast<cuuint64_t>(groups)};
        const cuuint64_t strides[3] = {pitch, 128, plane};
        const cuuint32_t box[4] = {64, box_rows, atoms, 1};
        r = fn(m, type, 4, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                    static_cast<cuuint64_t>(groups)};
        const cuuint64_t strides[2] = {pitch, plane};
        const cuuint32_t box[3] = {64, box_rows, 1};
        r = fn(m, type, 3, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    return r == CUDA_SUCCESS;
}

// Persistent grid: the clusters resident at once, never more than there can be tiles.
int gemm_grid(int64_t max_tiles) {
    int units = gemm_clusters();
    if (units <= 0) units = std::max(1, sm_count() / 2);
    return static_cast<int>(2 * std::max<int64_t>(1, std::min<int64_t>(units, max_tiles)));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Accumulator columns of a tile: 128 where even tiles of that width are no more
// than the clusters, else 256.  A 256-wide tile keeps the tensor cores and an
// SM's 64 bytes a clock from L2 equally busy; a narrower one is bound by the
// latter (1.6 times the time of a large product), but spreads a small product
// over more SMs.  Measured (us, 256 / 128 wide): gated, 4 experts x 128 rows of
// 4096 x 1024 26 / 22, one x 256 of 2048 x 704 14.2 / 12.7, 16 x 128 of
// 2048 x 1408 (176 tiles of 256) 44 / 48.
int pick_bn(int64_t tiles128) { return tiles128 <= std::max(1, gemm_clusters()) ? 128 : 256; }

ExpertGemmLaunch base_launch(int32_t W, int32_t e, int64_t A, int32_t dtype, const int32_t *recvCounts, int32_t *status) {
    ExpertGemmLaunch g;
    std::memset(&g, 0, sizeof g);
    g.recvCounts = recvCounts;
    g.W = W;
    g.e = e;
    g.A = static_cast<int32_t>(A);
    g.bf16 = dtype == A2AV_BF16;
    g.status = status;
    g.write_status = 1;
    g.wait_limit_ns = wait_limit_ns;
    return g;
}

// Tiles of the gradients, of bn accumulator columns: the rows expected, and the weights'.
int64_t row_tiles(int32_t e, int64_t A, int64_t H1, int64_t bn) {
    return A > 0 ? (ceil_div(A, 256) + e / 2) * ceil_div(H1, bn) : 0;
}
int64_t weight_tiles(int32_t e, int64_t H1, int64_t N, int phases, int64_t bn) {
    return e * ceil_div(H1, 256) * ceil_div(N, phases == 2 ? bn / 2 : bn);
}

// Slices of the gradients' contractions (see ExpertGemmLaunch): tiles that are
// few or far longer than the rest leave SMs idle, so their contraction is cut,
// and the slices' sums are joined by a second kernel.  Chosen by the blocks of
// the contraction that the fullest pair of SMs would go through, its tiles being
// dealt out in turn, plus the joining.  Measured (us, one slice / chosen): one
// expert, 8386 rows of 448 x 896 46 / 25, 16,384 of 1024 x 1024 103 / 58, 60,000
// of 256 x 256 289 / 41; 2 rows over 16 experts of 256 x 3456 27 / 18; 4 experts,
// 16,407 rows of 1024 x 4096 169 / 169 (not cut).  It depends on the shapes alone,
// since the workspace holds the sums.
// The choice hardly depends on the three costs: a third or twice kTileCost, and
// kJoinCost of 2 or 12, leave ten shapes' times as they are; half of kJoinBytes
// costs one of them (8386 of 448 x 896, 24.8 to 27.4), twice of it none.
constexpr double kTileCost = 3.0;       // of a tile beside its blocks, in blocks
constexpr double kJoinCost = 5.0;       // of the second kernel, in blocks
constexpr double kJoinBytes = 1.4e6;    // of sums written and read again in a block's time
struct Slices {
    int32_t rows, weights;
    size_t row_bytes, weight_bytes;  // of their sums
    size_t bytes() const { return row_bytes + weight_bytes; }
};
Slices slices_of(int32_t e, int64_t A, int64_t H1, int64_t N, int phases, int parts) {
    Slices best{1, 1, 0, 0};
    if (A == 0) return best;
    const int64_t bn = row_tiles(e, A, H1, 128) + weight_tiles(e, H1, N, phases, 128) <= kPairs ? 128 : 256;
    const int64_t tx = row_tiles(e, A, H1, bn), tw = weight_tiles(e, H1, N, phases, bn);
    const int64_t kx = ceil_div(N, 128), kw = ceil_div(A, static_cast<int64_t>(e) * 128);
    const double block = bn == 256 ? 1.0 : 0.75;
    double least = 0.0;
    for (int32_t sx = 1; sx <= std::min<int64_t>(kx, 16); sx *= 2)
        for (int32_t sw = 1; sw <= std::min<int64_t>(kw, 16); sw *= 2) {
            const Slices s{sx, sw, sx > 1 ? round256(static_cast<size_t>(sx) * A * H1 * 4) : 0,
                           sw > 1 ? round256(static_cast<size_t>(sw) * phases * e * H1 * N * 4) : 0};
            const double x = block * phases * parts * kx / sx + kTileCost, w = block * parts * kw / sw + kTileCost;
            const int64_t nx = tx * sx, n = nx + tw * sw;
            double cost = 0.0;
            for (const int64_t u : {int64_t{0}, nx % kPairs, (n + kPairs - 1) % kPairs}) {  // the fullest is one of these
                const int64_t mine = (n - u + kPairs - 1) / kPairs, mine_x = (std::max(nx - u, int64_t{0}) + kPairs - 1) / kPairs;
                cost = std::max(cost, mine_x * x + (mine - mine_x) * w);
            }
            if (s.bytes() > 0) cost += kJoinCost + s.bytes() / kJoinBytes;
            if (least == 0.0 || cost < least) least = cost, best = s;
        }
    return best;
}

// Gradients of one or two products with the same rows, in one launch:
// dX = sum_p D_p W_p^T, dW_p = X^T D_p.
// D: by product, then the second summands (parts 2).  sums: of the slices.
a2av_status run_gradients(ExpertGemmLaunch g, int phases, int parts, int64_t H1, int64_t N, const void *const D[4],
                          const void *X, const void *const Wt[2], void *dX, void *const dW[2], uint8_t *sums,
                          cudaStream_t stream) {
    const bool bf16 = g.bf16 != 0;
    g.grad = 1;
    g.phases = phases;
    g.parts = parts;
    g.one_a = g.one_b = N % 64 == 0;
    g.one_x = H1 % 64 == 0;
    const auto count = [&](int64_t bn, int64_t slices, int64_t w_slices) {
        return (dX ? slices * row_tiles(g.e, g.A, H1, bn) : 0) + (dW[0] ? w_slices * weight_tiles(g.e, H1, N, phases, bn) : 0);
    };
    const Slices s = slices_of(g.e, g.A, H1, N, phases, parts);
    g.slices = s.rows;
    g.w_slices = s.weights;
    g.part = reinterpret_cast<float *>(sums);
    g.part_w = reinterpret_cast<float *>(sums + s.row_bytes);
    g.bn = pick_bn(count(128, 1, 1));
    g.half_step = phases == 2 ? 0 : g.bn / 2;
    const uint32_t b_cols = g.bn / 2;  // columns of B a CTA stages
    for (int p = 0; p < phases * parts && g.A > 0; ++p)
        if (!operand_map(&g.tmA[p], D[p], 1, g.A, N, bf16, g.one_a) ||
            !operand_map(&g.tmD[p], D[p], 1, g.A, N, bf16, g.one_a, 128, b_cols / 64))
            return A2AV_ERR_CUDA;
    if (dX && g.A > 0) {
        g.K = static_cast<int32_t>(N);
        g.N = static_cast<int32_t>(H1);
        g.out = dX;
        for (int p = 0; p < phases; ++p)
            if (!operand_map(&g.tmB[p], Wt[p], g.e, H1, N, bf16, g.one_b, b_cols)) return A2AV_ERR_CUDA;
    }
    if (dW[0]) {
        g.wM = static_cast<int32_t>(H1);
        g.wN = static_cast<int32_t>(N);
        for (int i = 0; i < 2; ++i) g.out_w[i] = dW[phases == 2 ? i : 0];  // by accumulator half
        if (g.A > 0 && !operand_map(&g.tmX, X, 1, g.A, H1, bf16, g.one_x)) return A2AV_ERR_CUDA;
    }
    g.grid = gemm_grid(count(g.bn, s.rows, s.weights) + g.e * ceil_div(H1, g.bn) * s.rows);  // (without a tile the launch still stores the status)
    return a2av::launch_expert_gemm(g, stream) == cudaSuccess ? A2AV_OK : A2AV_ERR_CUDA;
}

a2av_status validate(const a2av_gated_desc *d) {
    if (!d) return A2AV_ERR_NULLPTR;
    if (d->W < 1 || d->e < 1 || d->e > a2av::kMaxExperts) return A2AV_ERR_INVALID;
    if (static_cast<int64_t>(d->W) * d->e > a2av::kMaxSegments) return A2AV_ERR_INVALID;
    if (d->H1 <= 0 || d->H1 >= 65536 || d->N <= 0 || d->N >= 65536) return A2AV_ERR_INVALID;
    if (d->A < 0 || d->A > INT32_MAX) return A2AV_ERR_INVALID;
    if (!type16(d->dtype)) return A2AV_ERR_INVALID;
    if (d->act != A2AV_ACT_SILU && d->act != A2AV_ACT_GELU_TANH) return A2AV_ERR_INVALID;
    // One source: the rows are expert-major already.  Several: the backward
    // pass reads permuteOut, so a call that saves for it writes it too.
    if (d->W == 1 ? d->want_permute_out != 0 : d->save && !d->want_permute_out) return A2AV_ERR_INVALID;
    if (!mult8(d->H1) || !mult8(d->N)) return A2AV_ERR_UNSUPPORTED;
    return A2AV_OK;
}

// Whether the weight-streaming kernel (gated_rows.cu) takes a forward call: the
// rows its fullest expert is expected to have fit one pass over the weights, or
// somewhat more where the tile kernel would have tiles for half of the SMs at
// most and a long way to go.
// Measured (us, streaming / tiles), rows an expert: 4 experts of 4096 x 1024
// from 8 sources, 16: 16 / 23, 32: 18 / 24, 64: 21 / 24, 96: 30 / 25, from one,
// 72: 21.2 / 21.8, 80: 28 / 22; 2 of 7168 x 2048, 72: 29 / 34, 80: 40 / 34; one
// of 7168 x 2048, 16: 14 / 32, 128: 18 / 33, 256: 31.8 / 32.7; one of 2048 x
// 704, 64: 10 / 12, 128: 12.3 / 12.6; 16 of 2048 x 1408, 16: 38 / 44, 32: 44 /
// 45, 64: 70 / 46; 4 of 2048 x 1024, 40: 12.5 / 13.9, 48: 14.4 / 13.9; 8 of 1032
// x 328 from 4, 40: 11.0 / 11.5, 48: 12.9 / 11.5.
// Rows are taken to spread at random.  Where they do not, the fullest expert's
// weights are read once for each pass (rows of it / all): 16 of 2048 x 1408,
// 128 / 512: 44 / 45, 512 / 512: 30 / 17; 32 of 4096 x 1536, 256 / 1024: 155 /
// 157, 512 / 1024: 163 / 156, 1024 / 1024: 79 / 28; 4 of 4096 x 1024, 128 / 128:
// 17 / 22.
bool few_rows(const a2av_gated_desc &d) {
    if (d.A == 0) return false;
    const double most = a2av::gated_rows_most(d.A, d.e);
    if (most <= 64.0) return true;
    if (d.H1 < 4096 || d.e * ((d.N + 127) / 128) >= 40) return false;
    return d.e == 1 ? d.A <= 256 : most <= 100.0;
}

size_t staged_bytes(const a2av_gated_desc *d) {
    return d->W > 1 && !d->want_permute_out ? round256(static_cast<size_t>(d->A) * d->H1 * 2) : 0;
}
// Counts of finished pieces of the slopes, by 128 rows.
size_t pieces_bytes(const a2av_gated_desc *d) {
    return d->save && d->A > 0 ? round256((static_cast<size_t>(d->A) / 128 + 1) * 4) : 0;
}
// Summands a slope is kept in.  One rounding to T adds as much to a gradient's
// error as the gradient's own rounding, however many rows or columns are summed
// (against float64, 1 to 1024 rows over 1 to 32 experts of 2048 x 1024: bf16
// 2.35e-3 with one summand, 1.66e-3 with two, which is the rounding of the exact
// gradient; fp16 2.94e-4 and 2.07e-4).  The second summand doubles what the
// tensor cores multiply and the stages they are fed (us, one / two, rows an
// expert: one expert of 2048 x 704, 1: 14 / 18, 32: 14 / 17, 256: 16 / 20; 4 of
// 4096 x 1024, 8: 41 / 61, 256: 54 / 85; 16 of 2048 x 1408, 1: 78 / 104, 32: 96 /
// 138, 256: 132 / 221).  So it is kept for calls of a few rows, where a user
// meets each row's error and it costs microseconds, and not for batches.
int slope_parts(const a2av_gated_desc *d) { return d->A <= 32 ? 2 : 1; }
size_t slope_bytes(const a2av_gated_desc *d) {  // one of dG, dU
    return d->save ? round256(static_cast<size_t>(d->A) * d->N * 2) : 0;
}

}  // namespace

extern "C" {

#ifdef A2AV_CHECKS
void a2av_checks_slopes_short(int32_t on, uint64_t limit_ns) {
    slopes_short = on != 0;
    wait_limit_ns = on ? limit_ns : kWaitLimitNs;
}
#endif

a2av_status a2av_rms_norm(const a2av_rms_norm_desc *desc, const void *x, const void *residual, const void *gamma,
                          void *h, void *y, void *codes, void *scales, float *rstd, a2av_stream_t stream) {
    if (!desc) return A2AV_ERR_NULLPTR;
    const a2av_rms_norm_desc &d = *desc;
    if (d.rows < 0 || d.rows > INT32_MAX || d.H <= 0 || d.H >= 65536 || !type16(d.dtype)) return A2AV_ERR_INVALID;
    if (!(d.eps >= 0.0f)) return A2AV_ERR_INVALID;
    if (d.x_stride < d.H || (residual && d.residual_stride != 0 && d.residual_stride < d.H)) return A2AV_ERR_INVALID;
    const a2av_status q = check_quant(d.qtype, d.qmode, d.H);
    if (q != A2AV_OK) return q;
    if (!mult8(d.H) || !mult8(d.x_stride) || (residual && !mult8(d.residual_stride))) return A2AV_ERR_UNSUPPORTED;
    if (!gamma || (d.rows > 0 && !x)) return A2AV_ERR_NULLPTR;
    if (d.rows > 0 && !h && !y && !codes && !rstd) return A2AV_ERR_NULLPTR;
    const a2av_status qo = check_quant_out(d.qtype, d.qmode, codes, scales, d.rows > 0);
    if (qo != A2AV_OK) return qo;
    for (const void *p : {x, residual, gamma, static_cast<const void *>(h), static_cast<const void *>(y)})
        if (!aligned(p, 16)) return A2AV_ERR_UNSUPPORTED;
    if (!aligned(rstd, 4)) return A2AV_ERR_UNSUPPORTED;
    if (d.rows == 0) return A2AV_OK;
    const int sms = sm_count();
    if (sms <= 0) return A2AV_ERR_CUDA;
    a2av::RmsNormLaunch p{static_cast<int32_t>(d.rows), static_cast<int32_t>(d.H), d.x_stride, d.residual_stride, x,
                          residual, gamma, h, y, static_cast<uint8_t *>(codes), scales, rstd, d.eps};
    return a2av::launch_rms_norm(p, d.dtype == A2AV_BF16, kind_of(d.qtype, d.qmode), sms,
                                 reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? A2AV_OK
               : A2AV_ERR_CUDA;
}

a2av_status a2av_rms_norm_backward_workspace_size(int64_t rows, int64_t H, int32_t dtype, size_t *bytes) {
    if (!bytes) return A2AV_ERR_NULLPTR;
    if (rows < 0 || rows > INT32_MAX || H <= 0 || H >= 65536 || !type16(dtype)) return A2AV_ERR_INVALID;
    if (!mult8(H)) return A2AV_ERR_UNSUPPORTED;
    const int blocks = a2av::rms_norm_grad_blocks(rows, H);
    *bytes = blocks > 1 ? round256(static_cast<size_t>(blocks) * H * 4) : 0;
    return A2AV_OK;
}

a2av_status a2av_rms_norm_backward(int64_t rows, int64_t H, int32_t dtype, const void *dy, const void *dh,
                                   const void *h, const void *gamma, const float *rstd, void *dx, float *dgamma,
                                   void *workspace, size_t workspace_bytes, a2av_stream_t stream) {
    size_t need = 0;
    const a2av_status s = a2av_rms_norm_backward_workspace_size(rows, H, dtype, &need);
    if (s != A2AV_OK) return s;
    if (rows > 0 && (!dy || !h || !gamma || !rstd || !dx)) return A2AV_ERR_NULLPTR;
    for (const void *p : {dy, dh, h, gamma, static_cast<const void *>(dx), static_cast<const void *>(dgamma)})
        if (!aligned(p, 16)) return A2AV_ERR_UNSUPPORTED;
    if (!aligned(rstd, 4)) return A2AV_ERR_UNSUPPORTED;
    if (dgamma && need > 0) {
        if (!workspace) return A2AV_ERR_NULLPTR;
        if (workspace_bytes < need || !aligned(workspace, 256)) return A2AV_ERR_WORKSPACE;
    }
    if (rows == 0 && !dgamma) return A2AV_OK;
    a2av::RmsNormGradLaunch p{static_cast<int32_t>(rows), static_cast<int32_t>(H), dy, dh, h, gamma, rstd, dx, dgamma,
                              static_cast<float *>(workspace), a2av::rms_norm_grad_blocks(rows, H)};
    return a2av::launch_rms_norm_grad(p, dtype == A2AV_BF16, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? A2AV_OK
               : A2AV_ERR_CUDA;
}

a2av_status a2av_glu_quant(const a2av_glu_desc *desc, const void *gate, const void *up, void *h, void *codes,
                           void *scales, a2av_stream_t stream) {
    if (!desc) return A2AV_ERR_NULLPTR;
    const a2av_glu_desc &d = *desc;
    if (d.rows < 0 || d.rows > INT32_MAX || d.N <= 0 || d.N >= 65536 || !type16(d.dtype)) return A2AV_ERR_INVALID;
    if (d.act != A2AV_ACT_SILU && d.act != A2AV_ACT_GELU_TANH) return A2AV_ERR_INVALID;
    if (d.stride < d.N) return A2AV_ERR_INVALID;
    const a2av_status q = check_quant(d.qtype, d.qmode, d.N);
    if (q != A2AV_OK) return q;
    if (!mult8(d.N) || !mult8(d.stride)) return A2AV_ERR_UNSUPPORTED;
    if (d.rows > 0 && (!gate || !up || (!h && !codes))) return A2AV_ERR_NULLPTR;
    const a2av_status qo = check_quant_out(d.qtype, d.qmode, codes, scales, d.rows > 0);
    if (qo != A2AV_OK) return qo;
    if (!aligned(gate, 16) || !aligned(up, 16) || !aligned(h, 16)) return A2AV_ERR_UNSUPPORTED;
    if (d.rows == 0) return A2AV_OK;
    a2av::GluLaunch p{d.rows, static_cast<int32_t>(d.N), d.stride, gate, up, h, static_cast<uint8_t *>(codes), scales,
                      0, 0};
    return a2av::launch_glu_quant(p, d.dtype == A2AV_BF16, d.act, kind_of(d.qtype, d.qmode),
                                  reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? A2AV_OK
               : A2AV_ERR_CUDA;
}

a2av_status a2av_gated_workspace_size(const a2av_gated_desc *desc, size_t *bytes) {
    if (!desc || !bytes) return A2AV_ERR_NULLPTR;
    const a2av_status s = validate(desc);
    if (s != A2AV_OK) return s;
    size_t back = 2 * slope_parts(desc) * slope_bytes(desc);
    if (desc->save) back += slices_of(desc->e, desc->A, desc->H1, desc->N, 2, slope_parts(desc)).bytes();
    *bytes = kStatusBytes + pieces_bytes(desc) + std::max(staged_bytes(desc), back);
    return A2AV_OK;
}

a2av_status a2av_gated_run(const a2av_gated_desc *desc, const void *ataOut, const int32_t *recvCounts,
                           const void *gateWeight, const void *upWeight, void *permuteOut, void *h, float *saved,
                           void *workspace, size_t workspace_bytes, a2av_stream_t stream_handle) {
    const a2av_status vs = validate(desc);
    if (vs != A2AV_OK) return vs;
    const a2av_gated_desc &d = *desc;
    if (!recvCounts || !gateWeight || !upWeight || !workspace) return A2AV_ERR_NULLPTR;
    if (d.A > 0 && (!ataOut || !h || (d.want_permute_out && !permuteOut) || (d.save && !saved)))
        return A2AV_ERR_NULLPTR;
    for (const void *p : {ataOut, gateWeight, upWeight, static_cast<const void *>(h),
                          static_cast<const void *>(d.want_permute_out ? permuteOut : nullptr)})
        if (!aligned(p, 16)) return A2AV_ERR_UNSUPPORTED;
    if (!aligned(recvCounts, 4) || (d.save && !aligned(saved, 32))) return A2AV_ERR_UNSUPPORTED;
    size_t need = 0;
    a2av_gated_workspace_size(desc, &need);
    if (workspace_bytes < need || !aligned(workspace, 256)) return A2AV_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const int sms = sm_count();
    if (sms <= 0) return A2AV_ERR_CUDA;

    if (few_rows(d)) {
        if (d.want_permute_out) {  // for the backward pass; this kernel gathers the rows itself, beside the permute
            const a2av::StageRowsLaunch sl{recvCounts, d.W,        d.e,
                                           static_cast<int32_t>(d.A), static_cast<int32_t>(d.H1),
                                           ataOut,     permuteOut, static_cast<int32_t *>(workspace)};
            if (a2av::launch_stage_rows(sl, sms, stream) != cudaSuccess) return A2AV_ERR_CUDA;
        }
        const bool bf16 = d.dtype == A2AV_BF16;
        a2av::GatedRowsLaunch r;
        std::memset(&r, 0, sizeof r);
        r.recvCounts = recvCounts;
        r.W = d.W;
        r.e = d.e;
        r.A = static_cast<int32_t>(d.A);
        r.K = static_cast<int32_t>(d.H1);
        r.N = static_cast<int32_t>(d.N);
        r.h = h;
        if (d.save) {
            r.saved[0] = saved;
            r.saved[1] = saved + d.A * d.N;
        }
        r.status = static_cast<int32_t *>(workspace);
        r.after_permute = d.want_permute_out;
        r.wait_limit_ns = wait_limit_ns;
        r.x = ataOut;
        if (!operand_map(&r.tmGate, gateWeight, d.e, d.H1, d.N, bf16, false) ||
            !operand_map(&r.tmUp, upWeight, d.e, d.H1, d.N, bf16, false))
            return A2AV_ERR_CUDA;
        return a2av::launch_gated_rows(r, bf16, d.act, stream) == cudaSuccess ? A2AV_OK : A2AV_ERR_CUDA;
    }
    ExpertGemmLaunch g = base_launch(d.W, d.e, d.A, d.dtype, recvCounts, static_cast<int32_t *>(workspace));
    const bool bf16 = g.bf16 != 0;
    g.act = d.act;
    g.K = static_cast<int32_t>(d.H1);
    g.N = static_cast<int32_t>(d.N);
    g.one_a = d.H1 % 64 == 0;
    g.one_b = d.N % 64 == 0;
    const auto count = [&](int64_t bn) { return (ceil_div(d.A, 256) + d.e / 2) * ceil_div(d.N, bn / 2); };
    g.bn = pick_bn(count(128));
    const void *rows = ataOut;
    if (d.W > 1 && d.A > 0) {
        // Expert-major rows: all of them, in permuteOut or the workspace, or only
        // those 128-row halves of a tile that straddle a (source, expert) run
        // boundary, the others being read in place.  (What has been staged is
        // read there: 463 us against 498 with whole runs read in place beside a
        // full permuteOut, 65,308 rows of 2048 x 1408.)
        void *dst = d.want_permute_out ? permuteOut
                                       : static_cast<uint8_t *>(workspace) + kStatusBytes + pieces_bytes(desc);
        g.direct_halves = !d.want_permute_out && d.A >= kLongRun * d.W * d.e;
        const a2av::PermuteLaunch pl{recvCounts, d.W, d.e, g.A, g.K, ataOut, dst, g.status, 1, 1, 8};
        const a2av::StageRowsLaunch sl{recvCounts, d.W, d.e, g.A, g.K, ataOut, dst, g.status};
        if ((g.direct_halves ? a2av::launch_permute(pl, sms, stream) : a2av::launch_stage_rows(sl, sms, stream)) !=
            cudaSuccess)
            return A2AV_ERR_CUDA;
        g.after_permute = 1;
        g.write_status = 0;
        rows = dst;
        if (g.direct_halves && !operand_map(&g.tmDirect, ataOut, 1, d.A, d.H1, bf16, g.one_a)) return A2AV_ERR_CUDA;
    }
    if (d.A > 0) {
        const uint32_t atoms = g.bn / 128;
        if (!operand_map(&g.tmA[0], rows, 1, d.A, d.H1, bf16, g.one_a) ||
            !operand_map(&g.tmB[0], gateWeight, d.e, d.H1, d.N, bf16, g.one_b, 128, atoms) ||
            !operand_map(&g.tmB[1], upWeight, d.e, d.H1, d.N, bf16, g.one_b, 128, atoms))
            return A2AV_ERR_CUDA;
        g.out = h;
        if (d.save) {
            g.saved[0] = saved;
            g.saved[1] = saved + static_cast<size_t>(d.A) * d.N;
        }
    }
    g.grid = gemm_grid((ceil_div(d.A, 256) + d.e) * ceil_div(d.N, g.bn / 2));
    return a2av::launch_expert_gemm(g, stream) == cudaSuccess ? A2AV_OK : A2AV_ERR_CUDA;
}

a2av_status a2av_gated_backward(const a2av_gated_desc *desc, const void *dh, const void *permuteOut,
                                const int32_t *recvCounts, const void *gateWeight, const void *upWeight,
                                const float *saved, void *dAtaOut, void *dGate, void *dUp, void *workspace,
                                size_t workspace_bytes, a2av_stream_t stream_handle) {
    const a2av_status vs = validate(desc);
    if (vs != A2AV_OK) return vs;
    const a2av_gated_desc &d = *desc;
    if (!d.save) return A2AV_ERR_INVALID;
    if (!recvCounts || !gateWeight || !upWeight || !workspace) return A2AV_ERR_NULLPTR;
    if (d.A > 0 && (!dh || !permuteOut || !saved)) return A2AV_ERR_NULLPTR;
    if ((dGate == nullptr) != (dUp == nullptr) || (d.A > 0 && !dAtaOut && !dGate)) return A2AV_ERR_NULLPTR;
    for (const void *p : {dh, permuteOut, gateWeight, upWeight, static_cast<const void *>(dAtaOut),
                          static_cast<const void *>(dGate), static_cast<const void *>(dUp)})
        if (!aligned(p, 16)) return A2AV_ERR_UNSUPPORTED;
    if (!aligned(recvCounts, 4) || !aligned(saved, 32)) return A2AV_ERR_UNSUPPORTED;
    size_t need = 0;
    a2av_gated_workspace_size(desc, &need);
    if (workspace_bytes < need || !aligned(workspace, 256)) return A2AV_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const int sms = sm_count();
    if (sms <= 0) return A2AV_ERR_CUDA;

    ExpertGemmLaunch g = base_launch(d.W, d.e, d.A, d.dtype, recvCounts, static_cast<int32_t *>(workspace));
    uint8_t *slopes = static_cast<uint8_t *>(workspace) + kStatusBytes + pieces_bytes(desc);
    const int parts = slope_parts(desc);
    void *const dG = slopes, *const dU = slopes + slope_bytes(desc);
    if (d.A > 0) {
        // (Without the rows' gradient the GEMM has nothing to do before all slopes
        // are there.)
        int32_t *pieces = nullptr;
        if (dAtaOut && slopes_beside(d.A, d.H1, d.N)) {
            pieces = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + kStatusBytes);
            if (cudaMemsetAsync(pieces, 0, pieces_bytes(desc), stream) != cudaSuccess) return A2AV_ERR_CUDA;
        }
        a2av::GluGradLaunch s{g.A, static_cast<int32_t>(d.N), dh, saved, saved + d.A * d.N, dG, dU, 0, pieces};
        if (parts == 2) s.low = 2 * slope_bytes(desc) / 16;
        if (a2av::launch_glu_grad(s, g.bf16, d.act, sms, stream) != cudaSuccess) return A2AV_ERR_CUDA;
        g.pieces = pieces;
        g.row_pieces = a2av::glu_grad_pieces(128, d.N);
        g.last_pieces = a2av::glu_grad_pieces(d.A % 128, d.N);
#ifdef A2AV_CHECKS
        if (slopes_short) ++g.row_pieces, ++g.last_pieces;
#endif
    }
    const void *const D[4] = {dG, dU, slopes + 2 * slope_bytes(desc), slopes + 3 * slope_bytes(desc)};
    const void *const Wt[2] = {gateWeight, upWeight};
    void *const dW[2] = {dGate, dUp};
    return run_gradients(g, 2, parts, d.H1, d.N, D, permuteOut, Wt, dAtaOut, dW, slopes + 2 * parts * slope_bytes(desc),
                         stream);
}

a2av_status a2av_gmm_backward_workspace_size(const a2av_gmm_desc *desc, size_t *bytes) {
    if (!desc || !bytes) return A2AV_ERR_NULLPTR;
    size_t unused = 0;
    const a2av_status s = a2av_gmm_workspace_size(desc, &unused);  // the shapes' limits
    if (s != A2AV_OK) return s;
    if (desc->BS != 0) return A2AV_ERR_INVALID;
    *bytes = kStatusBytes + slices_of(desc->e, desc->A, desc->H1, desc->N1, 1, 1).bytes();
    return A2AV_OK;
}

a2av_status a2av_gmm_backward(const a2av_gmm_desc *desc, const void *dY, const void *permuteOut,
                              const int32_t *recvCounts, const void *gmmWeight, void *dAtaOut, void *dWeight,
                              void *workspace, size_t workspace_bytes, a2av_stream_t stream_handle) {
    size_t need = 0;
    const a2av_status s = a2av_gmm_backward_workspace_size(desc, &need);
    if (s != A2AV_OK) return s;
    const a2av_gmm_desc &d = *desc;
    if (!recvCounts || !workspace) return A2AV_ERR_NULLPTR;
    if (d.A > 0 && (!dY || (!dAtaOut && !dWeight) || (dWeight && !permuteOut))) return A2AV_ERR_NULLPTR;
    if (dAtaOut && !gmmWeight) return A2AV_ERR_NULLPTR;
    for (const void *p : {dY, permuteOut, gmmWeight, static_cast<const void *>(dAtaOut),
                          static_cast<const void *>(dWeight)})
        if (!aligned(p, 16)) return A2AV_ERR_UNSUPPORTED;
    if (!aligned(recvCounts, 4)) return A2AV_ERR_UNSUPPORTED;
    if (workspace_bytes < need || !aligned(workspace, 256)) return A2AV_ERR_WORKSPACE;
    const ExpertGemmLaunch g = base_launch(d.W, d.e, d.A, d.dtype, recvCounts, static_cast<int32_t *>(workspace));
    const void *const D[4] = {dY, nullptr, nullptr, nullptr}, *const Wt[2] = {gmmWeight, nullptr};
    void *const dW[2] = {dWeight, nullptr};
    return run_gradients(g, 1, 1, d.H1, d.N1, D, permuteOut, Wt, dAtaOut, dW,
                         static_cast<uint8_t *>(workspace) + kStatusBytes, reinterpret_cast<cudaStream_t>(stream_handle));
}

}  // extern "C"
