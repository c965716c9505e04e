// Waits, signals and copies of the operators beside the layer's own kernels, on the wrappers of sm100.cuh and the bounded waits of
// common.cuh.
#pragma once
#include "common.cuh"

namespace moe {

// As mbar_try_wait, but the thread may be suspended for up to `ns` nanoseconds while the phase is incomplete.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar_addr, uint32_t parity, uint32_t ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar_addr), "r"(parity), "r"(ns)
        : "memory");
    return ok != 0;
}

// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar_addr, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar_addr), "r"(parity)
        : "memory");
    return ok != 0;
}

// True in one lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(e));
    return e != 0;
}

// Untiled copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) from global to this CTA's shared memory; completion
// is signalled on `bar` as transaction bytes.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// As mbar_arrive_cluster without cluster-scope release semantics (which cost a memory barrier of about 2000 cycles): for signals that order
// nothing but this thread's completed tensor-memory loads (tcgen05.wait::ld, then tcgen05.fence::before_thread_sync).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Store 16 bytes into a CTA of the cluster (addresses of mapa_shared): counted on its barrier as transaction bytes.
__device__ __forceinline__ void store_remote(uint32_t cluster_addr, const float4& v, uint32_t cluster_bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(cluster_addr),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(cluster_bar)
                 : "memory");
}

// As mbar_wait_bounded, for waits once per K block on several roles' critical paths: the limit is the caller's (read once, by
// wait_limit_ns() at the kernel's start; reading it in the wait costs an L2 access each time the barrier is not ready), the clock
// is looked at only after a first poll, and each poll sleeps in hardware for up to 20 us instead of spinning. The limit is a value, or
// where it lies in shared memory (for kernels that have no two registers for it).
__device__ __forceinline__ uint64_t limit_of(uint64_t limit) { return limit; }
__device__ __forceinline__ uint64_t limit_of(const volatile uint64_t* limit) { return *limit; }
template <typename Limit>
__device__ __forceinline__ bool mbar_wait_within(uint64_t* bar, uint32_t parity, volatile int* abort_flag, Limit limit) {
    const uint32_t addr = smem_u32(bar);
    if (mbar_try_wait_for(addr, parity, 20000)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_for(addr, parity, 20000)) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > limit_of(limit)) {
            *abort_flag = 1;
            flag_error(MOE_DEVERR_WAIT_TIMEOUT);
            return false;
        }
    }
}

}  // namespace moe
