// CTA-pair building blocks (cluster of two, tcgen05 cta_group::2) of the
// expert-layer GEMMs: barriers across the pair, TMA loads that complete on
// the even CTA's barrier, MMA issue and TMEM allocation for both CTAs.
#pragma once

#include <cstdint>

#include "plan.cuh"
#include "ptx.cuh"

namespace a2av {
namespace pair {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The same after reads only (of TMEM, or of another CTA's shared memory, their
// values used or waited for): it does not hold the arrival back until this
// thread's stores to global memory have been seen by the cluster, which costs an
// epilogue more than the stores.
__device__ __forceinline__ void arrive_reads_done(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait on an mbarrier phase, acquiring at cluster scope (arrivals may
// come from the peer CTA).  False: gave up, or another role did; the abort
// flag and the status word are set.
static __device__ __noinline__ bool wait_phase(int32_t *abort_flag, uint32_t bar, uint32_t parity, int32_t *status,
                                        uint64_t limit_ns) {
    if (try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        for (int i = 0; i < 64; ++i)
            if (try_wait_cluster(bar, parity)) return true;
        if (*reinterpret_cast<volatile int32_t *>(abort_flag)) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            *reinterpret_cast<volatile int32_t *>(abort_flag) = 1;
            atomicOr(status, kStatusTimeout);
            return false;
        }
    }
}

// The same by a whole warp: its lanes try and give up one by one, so the phase may
// complete between one lane's last try and another's next.  They leave with one
// answer, since what follows (votes, tcgen05 loads, the cluster's barrier) needs
// the whole warp.
__device__ __forceinline__ bool wait_phase_warp(int32_t *abort_flag, uint32_t bar, uint32_t parity, int32_t *status,
                                                uint64_t limit_ns) {
    return __all_sync(0xffffffffu, wait_phase(abort_flag, bar, parity, status, limit_ns));
}

// After a wait was given up: a millisecond for the copies and products still in
// flight, which take microseconds, before shared memory and TMEM are given back.
static __device__ __noinline__ void let_settle() {
    const uint64_t t0 = global_timer_ns();
    for (int i = 0; i < 100000 && global_timer_ns() - t0 < 1000000; ++i) __nanosleep(1000);
}

// TMA loads whose barrier may live in the peer CTA.
__device__ __forceinline__ void load_3d(uint32_t dst, const void *tmap, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void load_4d(uint32_t dst, const void *tmap, uint32_t bar, int32_t x, int32_t y, int32_t z,
                                        int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                    uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One arrival on the barrier at this offset in both CTAs when this thread's
// earlier tcgen05 operations have completed.
__device__ __forceinline__ void commit(uint32_t bar) {
    const uint16_t both = 3;
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"(both)
        : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free_pair(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

}  // namespace pair
}  // namespace a2av
