// Device-side building blocks that the paged kernels use beside saga_device.cuh.
#pragma once

#include "saga_device.cuh"

namespace saga {

// Takes a ticket: the block's writes before it (ordered by a block barrier)
// are visible to whoever takes a later one, and theirs to this block after the
// next barrier (read through L2).  Returns the tickets taken before.
__device__ __forceinline__ uint32_t take_ticket(uint32_t* counter) {
    uint32_t n;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
    return n;
}

// Adds to the bytes that the barrier's current phase waits for.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
}

// Arrives for the current phase and leaves the barrier: later phases expect one arrival fewer.
__device__ __forceinline__ void mbar_arrive_drop(uint64_t* bar) {
    asm volatile("mbarrier.arrive_drop.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

}  // namespace saga
