// C ABI of the expert layer for a few tokens (declared in include/a2av_moe.h):
// argument checks, tensor maps, launches.
#include <cmath>
#include <cstring>

#include "a2av_moe.h"
#include "moe.h"
#include "tensor_map.h"

namespace {

constexpr size_t kStatusBytes = 256;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // bound on every device-side wait

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// [groups][rows][cols]: boxes of 64 columns x box_rows rows x box_groups, 128-byte swizzled.
bool tile_map(CUtensorMap *m, const void *ptr, int64_t groups, int64_t rows, int64_t cols, bool bf16, int box_rows,
              int box_groups) {
    auto fn = a2av::tensor_map_encode();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(groups)};
    const cuuint64_t pitch = static_cast<cuuint64_t>(cols) * 2;
    const cuuint64_t strides[2] = {pitch, groups > 1 ? pitch * rows : pitch};  // (the second is not used with one group)
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_groups)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(ptr),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

a2av_status validate(const a2av_moe_desc *d) {
    if (!d) return A2AV_ERR_NULLPTR;
    if (d->T < 0 || d->T > a2av::kMoeTokens || d->E < 1 || d->E > a2av::kMoeExperts) return A2AV_ERR_INVALID;
    if (d->K < 1 || d->K > a2av::kMoeChosen || d->K > d->E) return A2AV_ERR_INVALID;
    if (d->H <= 0 || d->H >= 65536 || d->N <= 0 || d->N >= 65536) return A2AV_ERR_INVALID;
    if (d->dtype != A2AV_BF16 && d->dtype != A2AV_FP16) return A2AV_ERR_INVALID;
    if (d->router_dtype != d->dtype && d->router_dtype != A2AV_FP32) return A2AV_ERR_INVALID;
    if (d->act != A2AV_ACT_SILU && d->act != A2AV_ACT_GELU_TANH) return A2AV_ERR_INVALID;
    if (d->score != A2AV_SCORE_SOFTMAX && d->score != A2AV_SCORE_SIGMOID) return A2AV_ERR_INVALID;
    if (!std::isfinite(d->scale)) return A2AV_ERR_INVALID;
    if (d->H % 8 != 0 || d->N % 8 != 0) return A2AV_ERR_UNSUPPORTED;
    return A2AV_OK;
}

size_t logit_bytes(const a2av_moe_desc &d) { return round256(static_cast<size_t>(d.T) * d.E * 4); }
size_t chosen_bytes(const a2av_moe_desc &d) { return round256(static_cast<size_t>(d.T) * d.K * sizeof(int2)); }
constexpr size_t kArrivalBytes = 2 * a2av::kMoeCtas * 4;
// Shares of jobs; the second product's, half as large, take the place of the first's.
size_t sum_bytes(const a2av_moe_desc &d) { return static_cast<size_t>(a2av::kMoeCtas) * 2 * d.T * 1024; }
size_t value_bytes(const a2av_moe_desc &d) { return round256(static_cast<size_t>(d.T) * d.K * d.N * 4); }

size_t workspace_bytes_of(const a2av_moe_desc &d) {
    return kStatusBytes + round256(kArrivalBytes) + logit_bytes(d) + chosen_bytes(d) + value_bytes(d) +
           sum_bytes(d);
}

}  // namespace

extern "C" {

a2av_status a2av_moe_workspace_size(const a2av_moe_desc *desc, size_t *bytes) {
    if (!desc || !bytes) return A2AV_ERR_NULLPTR;
    const a2av_status s = validate(desc);
    if (s != A2AV_OK) return s;
    *bytes = workspace_bytes_of(*desc);
    return A2AV_OK;
}

a2av_status a2av_moe_run(const a2av_moe_desc *desc, const void *x, const void *router, const float *bias,
                         const void *gate, const void *up, const void *down, const void *residual, void *y,
                         int32_t *experts, float *weights, void *workspace, size_t workspace_bytes,
                         a2av_stream_t stream_handle) {
    const a2av_status vs = validate(desc);
    if (vs != A2AV_OK) return vs;
    const a2av_moe_desc &d = *desc;
    if (!router || !gate || !up || !down || !workspace || (d.T > 0 && (!x || !y))) return A2AV_ERR_NULLPTR;
    for (const void *p : {x, router, static_cast<const void *>(bias), gate, up, down, residual, static_cast<const void *>(y)})
        if (!aligned(p, 16)) return A2AV_ERR_UNSUPPORTED;
    if (!aligned(experts, 4) || !aligned(weights, 4)) return A2AV_ERR_UNSUPPORTED;
    if (workspace_bytes < workspace_bytes_of(d) || !aligned(workspace, 256))
        return A2AV_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const bool bf16 = d.dtype == A2AV_BF16;
    uint8_t *const arrivals = static_cast<uint8_t *>(workspace) + kStatusBytes;
    uint8_t *const logits = arrivals + round256(kArrivalBytes), *const chosen = logits + logit_bytes(d);
    uint8_t *const values = chosen + chosen_bytes(d);

    a2av::MoeRouterLaunch r{d.T, d.E, static_cast<int32_t>(d.H), x, router, reinterpret_cast<float *>(logits),
                            static_cast<int32_t *>(workspace), reinterpret_cast<int32_t *>(arrivals)};
    a2av::MoeRowsLaunch g;
    std::memset(&g, 0, sizeof g);
    g.choice = a2av::MoeChoice{d.T, d.E, d.K, d.score, d.renormalise != 0, d.scale, r.logits, bias, experts, weights,
                                reinterpret_cast<int2 *>(chosen)};
    g.H = static_cast<int32_t>(d.H);
    g.N = static_cast<int32_t>(d.N);
    g.residual = residual;
    g.h = values;
    g.sums = reinterpret_cast<float *>(values + value_bytes(d));
    g.arrivals = r.arrivals;
    g.y = y;
    g.status = r.status;
    g.wait_limit_ns = kWaitLimitNs;
    a2av::MoeRowsLaunch o = g;
    o.arrivals += a2av::kMoeCtas;
    o.units = r.status + 1;
    if (d.T > 0 && (!tile_map(&g.tmA[0], gate, d.E, d.H, d.N, bf16, 64, 1) ||
                    !tile_map(&g.tmA[1], up, d.E, d.H, d.N, bf16, 64, 1) ||
                    !tile_map(&g.tmX, x, 1, d.T, d.H, bf16, a2av::moe_unit_rows(d.T, d.E, d.K, false), 1) ||
                    !tile_map(&o.tmA[0], down, d.E, d.N, d.H, bf16, 64, 1) ||
                    !tile_map(&o.tmX, g.h, 2, d.T * d.K, d.N, bf16, a2av::moe_unit_rows(d.T, d.E, d.K, true), 2)))
        return A2AV_ERR_CUDA;
    if (a2av::launch_moe_router(r, bf16, d.router_dtype == A2AV_FP32, stream) != cudaSuccess) return A2AV_ERR_CUDA;
    if (d.T == 0) return A2AV_OK;  // (the status is stored)
    if (a2av::launch_moe_choose(g.choice, stream) != cudaSuccess) return A2AV_ERR_CUDA;
    if (a2av::launch_moe_gated(g, bf16, d.act, stream) != cudaSuccess) return A2AV_ERR_CUDA;
    return a2av::launch_moe_down(o, bf16, stream) == cudaSuccess ? A2AV_OK : A2AV_ERR_CUDA;
}

}  // extern "C"
