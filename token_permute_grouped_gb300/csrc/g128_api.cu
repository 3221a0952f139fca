// C ABI of the grouped product of 8-bit rows with a float32 scale per 128
// (declared in include/a2av_gmm_g128.h): argument checks, tensor maps, launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "a2av_gmm_g128.h"
#include "ffn.h"
#include "g128.h"
#include "kernels.h"
#include "per_device.h"
#include "plan.cuh"
#include "tensor_map.h"

namespace {

constexpr size_t kStatusBytes = 256;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // bound on every device-side wait

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Device {
    int sms, clusters;
};
const Device *device_of() {
    static a2av::PerDevice<Device> cache;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
    return cache.get(dev, [dev](Device &d) {
        return cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
               (d.clusters = a2av::g128_gemm_max_clusters()) > 0;
    });
}

// Codes [groups][rows][K]: boxes of 128 codes x box_rows rows, 128-byte swizzled.
bool codes_map(CUtensorMap *m, const void *ptr, int64_t groups, int64_t rows, int64_t K, uint32_t box_rows) {
    auto fn = a2av::tensor_map_encode();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(groups)};
    const cuuint64_t pitch = static_cast<cuuint64_t>(K);
    const cuuint64_t strides[2] = {pitch, groups > 1 ? pitch * rows : pitch};  // (the second is not used with one group)
    const cuuint32_t box[3] = {128, box_rows, 1}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

a2av_status validate(const a2av_gmm_g128_desc *d) {
    if (!d) return A2AV_ERR_NULLPTR;
    if (d->W < 1 || d->e < 1 || d->e > a2av::kMaxExperts) return A2AV_ERR_INVALID;
    if (static_cast<int64_t>(d->W) * d->e > a2av::kMaxSegments) return A2AV_ERR_INVALID;
    if (d->H1 <= 0 || d->H1 >= 65536 || d->N1 <= 0 || d->N1 >= 65536) return A2AV_ERR_INVALID;
    if (d->A < 0 || d->A > INT32_MAX) return A2AV_ERR_INVALID;
    if (d->dtype != A2AV_BF16 && d->dtype != A2AV_FP16) return A2AV_ERR_INVALID;
    if (d->qtype != A2AV_Q_E4M3FN && d->qtype != A2AV_Q_E5M2) return A2AV_ERR_INVALID;
    if (d->H1 % 128 != 0 || d->N1 % 8 != 0) return A2AV_ERR_UNSUPPORTED;
    return A2AV_OK;
}

// Whether the weight-streaming kernel (g128_rows.cu) takes a call: the rows of the
// fullest expert, if they spread at random, fit one pass over the weights, and the
// weights of the experts that they reach are long to read.
// Measured (us, streaming / tiles, weights from HBM; rows over experts of H1 x N1):
// 1 over 1 of 7168 x 4096 14.6 / 23.9, 8 over 4 of 4096 x 2048 15.4 / 17.5, 16 over
// 4 19.4 / 23.3, 8 over 16 of 2048 x 2816 17.4 / 18.5, 32 over 16 27 / 32, 64 over
// 32 of 4096 x 1536 50 / 54, 16 over 1 of 4096 x 2048 12.6 / 13.4; less to read: 8
// over 1 of 2048 x 2048 10.2 / 8.6, 1 over 1 of 1024 x 1024 7.9 / 6.0.  More rows at
// a time: 32 over 1 of 7168 x 4096 20.4 / 20.5, 64 over 4 of 4096 x 2048 20.5 / 17.5,
// 128 over 4 28 / 17.5 (a warp's 64 sums and their exchange cost more than the padded
// rows of a tile).
bool few_rows(const a2av_gmm_g128_desc &d) {
    if (d.A == 0 || a2av::gated_rows_most(d.A, d.e) > a2av::kG128UnitRows) return false;
    const double reached = d.e * (1.0 - std::pow(1.0 - 1.0 / d.e, static_cast<double>(d.A)));
    return reached * d.H1 * d.N1 >= 8e6;
}
// Behind the status, for few rows: arrivals, shares of sums, the rows' scales; then
// the staged rows.
constexpr size_t kArrivalBytes = (a2av::kG128Ctas * 4 + 255) / 256 * 256;
constexpr size_t kSumBytes = static_cast<size_t>(a2av::kG128Ctas) * 2 * a2av::kG128UnitRows * 128 * 4;
size_t scale_bytes(const a2av_gmm_g128_desc &d) { return round256(static_cast<size_t>(d.A) * (d.H1 / 128) * 4); }
size_t few_bytes(const a2av_gmm_g128_desc &d) { return few_rows(d) ? kArrivalBytes + kSumBytes + scale_bytes(d) : 0; }

size_t staged_bytes(const a2av_gmm_g128_desc *d) {
    return d->W > 1 ? round256(static_cast<size_t>(d->A) * d->H1) : 0;
}

// Mean rows of a (source, expert) run from which whole halves are read in place (us, in
// place / all copied, medians of ten: 8 sources, 8 experts of 2048 x 2816, runs of 64: 35 /
// 33.5, 96: 53 / 49, 128: 70 / 69, 160: 82 / 81, 192: 89 / 87, 256: 111 / 109; 16 sources, 8
// of 4096 x 2048, 128: 150 / 154; 4 of 4096 x 4096, 192: 195 / 200; 8 of 7168 x 2048, 256:
// 224 / 242; 8 of 7168 x 4096, 32 sources, 135: 827 / 814, 8 sources, 539: 764 / 812).
constexpr int64_t kLongRun = 192;

}  // namespace

extern "C" {

a2av_status a2av_gmm_g128_workspace_size(const a2av_gmm_g128_desc *desc, size_t *bytes) {
    if (!desc || !bytes) return A2AV_ERR_NULLPTR;
    const a2av_status s = validate(desc);
    if (s != A2AV_OK) return s;
    *bytes = kStatusBytes + few_bytes(*desc) + staged_bytes(desc);
    return A2AV_OK;
}

a2av_status a2av_gmm_g128_run(const a2av_gmm_g128_desc *desc, const void *ataOut_q, const float *ataOut_s,
                              const int32_t *recvCounts, const void *gmmWeight_q, const float *gmmWeight_s, void *gmmY,
                              void *workspace, size_t workspace_bytes, a2av_stream_t stream_handle) {
    const a2av_status vs = validate(desc);
    if (vs != A2AV_OK) return vs;
    const a2av_gmm_g128_desc &d = *desc;
    if (!recvCounts || !gmmWeight_q || !gmmWeight_s || !workspace) return A2AV_ERR_NULLPTR;
    if (d.A > 0 && (!ataOut_q || !ataOut_s || !gmmY)) return A2AV_ERR_NULLPTR;
    for (const void *p : {ataOut_q, gmmWeight_q, static_cast<const void *>(gmmY)})
        if (!aligned(p, 16)) return A2AV_ERR_UNSUPPORTED;
    for (const void *p : {static_cast<const void *>(ataOut_s), static_cast<const void *>(gmmWeight_s),
                          static_cast<const void *>(recvCounts)})
        if (!aligned(p, 4)) return A2AV_ERR_UNSUPPORTED;
    size_t need = 0;
    a2av_gmm_g128_workspace_size(desc, &need);
    if (workspace_bytes < need || !aligned(workspace, 256)) return A2AV_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const Device *dev = device_of();
    if (!dev) return A2AV_ERR_CUDA;
    const bool bf16 = d.dtype == A2AV_BF16;

    a2av::G128Launch g;
    std::memset(&g, 0, sizeof g);
    g.recvCounts = recvCounts;
    g.W = d.W;
    g.e = d.e;
    g.A = static_cast<int32_t>(d.A);
    g.K = static_cast<int32_t>(d.H1);
    g.N = static_cast<int32_t>(d.N1);
    g.qtype = d.qtype;
    g.xs = ataOut_s;
    g.ws = gmmWeight_s;
    g.y = gmmY;
    g.status = static_cast<int32_t *>(workspace);
    g.write_status = 1;
    g.wait_limit_ns = kWaitLimitNs;
    uint8_t *const arrivals = static_cast<uint8_t *>(workspace) + kStatusBytes, *const staged = arrivals + few_bytes(d);
    if (few_rows(d)) {
        void *const dst = d.W > 1 ? staged : nullptr;  // (from one source the rows are expert-major as they arrive)
        g.arrivals = reinterpret_cast<int32_t *>(arrivals);
        g.sums = reinterpret_cast<float *>(arrivals + kArrivalBytes);
        float *const scales = reinterpret_cast<float *>(arrivals + kArrivalBytes + kSumBytes);
        g.xs = scales;
        const a2av::G128Stage st{recvCounts, d.W, d.e, g.A, g.K, ataOut_q, ataOut_s, dst, scales, g.status, g.arrivals};
        if (!codes_map(&g.tmA, dst ? dst : ataOut_q, 1, d.A, d.H1, a2av::kG128UnitRows) ||
            !codes_map(&g.tmB, gmmWeight_q, d.e, d.N1, d.H1, 128))
            return A2AV_ERR_CUDA;
        if (a2av::launch_g128_stage(st, stream) != cudaSuccess) return A2AV_ERR_CUDA;
        return a2av::launch_g128_rows(g, bf16, stream) == cudaSuccess ? A2AV_OK : A2AV_ERR_CUDA;
    }
    const int64_t strips = ceil_div(d.N1, 128);
    // Waves of single CTAs' tiles and of pairs', each expert's last tile half full: a
    // pair's takes 1.5 times as long for four times the work (us, single / pairs: 128 rows
    // of 1024 x 1024 5.5 / 8.2, 512 of 2048 x 2048 8.4 / 12.5, 300 over 4 experts of 4096 x
    // 2048 15 / 20, 1634 over 16 of 2048 x 2816 29 / 35, 1000 over 32 of 4096 x 1536 48 /
    // 54; 2048 over 4 of 2048 x 1408 21 / 18, 4096 over 8 of 2048 x 2816 48 / 37, 16,384 over
    // 8 143 / 114).
    const int64_t single = ceil_div((ceil_div(d.A, 128) + d.e / 2) * strips, dev->sms);
    const int64_t pairs = ceil_div((ceil_div(d.A, 256) + d.e / 2) * ceil_div(strips, 2), dev->clusters);
    g.pair = 2 * single >= 3 * pairs;
    const void *rows = ataOut_q;
    if (d.W > 1 && d.A > 0) {
        // Expert-major rows: all of them, or only the 128-row halves of a tile that
        // straddle a run's end, the others being read in place.  (The copies take the
        // rows as 16-bit elements.)
        void *dst = staged;
        g.direct_halves = d.A >= kLongRun * d.W * d.e;
        const a2av::PermuteLaunch pl{recvCounts, d.W, d.e, g.A, g.K / 2, ataOut_q, dst, g.status, 1, 1, 8};
        const a2av::StageRowsLaunch sl{recvCounts, d.W, d.e, g.A, g.K / 2, ataOut_q, dst, g.status};
        if ((g.direct_halves ? a2av::launch_permute(pl, dev->sms, stream) : a2av::launch_stage_rows(sl, dev->sms, stream)) !=
            cudaSuccess)
            return A2AV_ERR_CUDA;
        g.after_permute = 1;
        g.write_status = 0;
        rows = dst;
        if (g.direct_halves && !codes_map(&g.tmDirect, ataOut_q, 1, d.A, d.H1, 128)) return A2AV_ERR_CUDA;
    }
    if (d.A > 0 && (!codes_map(&g.tmA, rows, 1, d.A, d.H1, 128) ||
                    !codes_map(&g.tmB, gmmWeight_q, d.e, d.N1, d.H1, 128)))
        return A2AV_ERR_CUDA;
    // (At most one tile more an expert than its rows fill.)
    const int64_t tiles = g.pair ? (ceil_div(d.A, 256) + d.e) * ceil_div(strips, 2) : (ceil_div(d.A, 128) + d.e) * strips;
    const int64_t units = std::max<int64_t>(1, std::min<int64_t>(g.pair ? dev->clusters : dev->sms, tiles));
    g.grid = static_cast<int32_t>(g.pair ? 2 * units : units);
    return a2av::launch_g128_gemm(g, bf16, stream) == cudaSuccess ? A2AV_OK : A2AV_ERR_CUDA;
}

}  // extern "C"
