// Asynchronous copies of a word of 16 or 8 bytes into a shared-memory slot of the
// thread that issues them, visible to it once the group that holds the copy is
// waited for. No other thread reads the slot, so no barrier is needed.
#pragma once

#include "common.cuh"

namespace rmsn {

template <int BYTES>
__device__ __forceinline__ bool slot_in(uint32_t slot) {
    const uint32_t b = smem_u32(rmsn_dynamic_smem);
    return slot >= b && slot - b + BYTES <= dynamic_smem_bytes();
}
template <int BYTES = 16>
__device__ __forceinline__ void copy_own(uint32_t slot, const void* src, int* status) {
    static_assert(BYTES == 16 || BYTES == 8, "the asynchronous copies in use");
    if (!RMSN_OK(slot_in<BYTES>(slot), status)) return;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(slot), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 ld_slot(uint32_t slot) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(slot)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_slot_8(uint32_t slot) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(slot) : "memory");
    return v;
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

}  // namespace rmsn
