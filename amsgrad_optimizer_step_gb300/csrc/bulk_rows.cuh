// Rows on their way from global to shared memory as bulk copies, which one thread issues and an
// mbarrier a row completes.  Every wait is bounded (about a second).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fa {

constexpr uint32_t kRowWaitTries = 1u << 20;  // of at most kRowWaitNs each
constexpr uint32_t kRowWaitNs = 1000;

__device__ __forceinline__ uint32_t shared_address(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void row_barrier_init(uint64_t *bar) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_address(bar)) : "memory");
}
// After the inits, before the first copy.
__device__ __forceinline__ void row_barriers_ready() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// Ordinary writes to memory that copies will write later, by every thread that made them.
__device__ __forceinline__ void shared_writes_before_copies() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void row_expect(uint64_t *bar, uint32_t bytes) {
    asm volatile("{\n .reg .b64 st;\n mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}"
                 ::"r"(shared_address(bar)), "r"(bytes) : "memory");
}
// 16-byte aligned on both sides, a multiple of 16 bytes.
__device__ __forceinline__ void row_copy(void *dst, const void *src, uint32_t bytes,
                                         uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(shared_address(dst)), "l"(src), "r"(bytes), "r"(shared_address(bar)) : "memory");
}
// False where the copies did not arrive in time.
__device__ __forceinline__ bool row_wait(uint64_t *bar, uint32_t parity) {
    for (uint32_t i = 0; i < kRowWaitTries; ++i) {
        uint32_t ok;
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
                     " selp.u32 %0, 1, 0, p;\n}"
                     : "=r"(ok) : "r"(shared_address(bar)), "r"(parity), "r"(kRowWaitNs) : "memory");
        if (ok) return true;
    }
    return false;
}

}  // namespace fa
