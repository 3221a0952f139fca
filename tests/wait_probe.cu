// One warp waits on an mbarrier in shared memory, half of its lanes for a phase that has completed and half for one that
// never will; out[lane] is each lane's answer.  (Built and called by test_gpu_ffn_waits.py.)
#include "pair.cuh"

namespace {

__global__ void probe(int32_t *out, int32_t *status, uint64_t limit_ns) {
    __shared__ uint64_t bar;
    __shared__ int32_t abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        a2av::mbar_init(a2av::smem_u32(&bar), 1);
        a2av::fence_barrier_init();
    }
    __syncthreads();
    // A fresh barrier: the phase of parity 1 counts as completed, that of parity 0 is under way.
    const uint32_t parity = threadIdx.x < 16 ? 1 : 0;
    out[threadIdx.x] = a2av::pair::wait_phase_warp(&abort_flag, a2av::smem_u32(&bar), parity, status, limit_ns);
    __syncwarp();
    out[32 + threadIdx.x] = a2av::pair::wait_phase_warp(&abort_flag, a2av::smem_u32(&bar), 1, status, limit_ns);
}

}  // namespace

extern "C" int run_probe(int32_t *out, int32_t *status, uint64_t limit_ns, cudaStream_t stream) {
    probe<<<1, 32, 0, stream>>>(out, status, limit_ns);
    return cudaGetLastError();
}
