// Loads from a buffer straight into LDS, and the waits and barrier around them.
#pragma once

#include "moe_device.h"

namespace moeq4 {

typedef __amdgpu_buffer_rsrc_t buf_rsrc_t;
typedef __attribute__((address_space(3))) void* lds_dst_t;

// Buffer of `bytes` bytes: a load at or past its end returns zeros without touching
// memory.  The builtins exist only in the device pass.
__device__ __forceinline__ buf_rsrc_t make_buf(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

// 16 bytes per lane: lane l writes lds + 16 l (lds uniform over the wave).  The buffer's bound holds
// for voff alone: where a load may pass the end, voff does so without soff.
__device__ __forceinline__ void buf_to_lds16(buf_rsrc_t r, void* lds, uint32_t voff, uint32_t soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_dst_t)lds, 16, voff, soff, 0, 0);
#endif
}

// 16 bytes per lane into registers.
__device__ __forceinline__ u32x4_t buf_load16_u(buf_rsrc_t r, uint32_t voff, uint32_t soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
#else
    return u32x4_t{0, 0, 0, 0};
#endif
}

// Waits until at most N of this wave's vector loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Waits for this wave's accesses of LDS.
__device__ __forceinline__ void wait_lds() {
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));
}

// Workgroup barrier without a memory fence, which would wait for every load still in
// flight: the caller has waited for what the other waves must see.  Nothing moves
// across it.
__device__ __forceinline__ void bare_barrier_i8() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

}  // namespace moeq4
