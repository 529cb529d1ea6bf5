// Direct loads into the LDS and the waits that belong to them.
#pragma once

#include "moe_internal.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Direct buffer -> LDS load of 16 bytes per lane from `base` + `off` (zeros from
// `bytes` on): lane l's bytes land at dst + 16 l (dst is uniform across the wave).
// ONCE: a non-temporal load, for lines that are read once.
template <bool ONCE>
__device__ __forceinline__ void buffer_load_lds16(const void* base, uint32_t bytes, uint32_t off, void* dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00020000),
                                             (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, ONCE ? 2 : 0);
}

// Byte offset that lies behind every buffer (their extents are checked on the
// host to be at most this): loads there return zeros.
constexpr uint32_t kOutOfRange = 0xFFFF0000u;

// s_waitcnt until no LDS operation and at most N vector-memory operations of this wave are
// outstanding, then the workgroup barrier.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The workgroup barrier once this wave's LDS operations are done (loads into the
// LDS may still be on their way).
__device__ __forceinline__ void wait_lds_and_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Reads of 16 bytes per lane at LDS byte addresses, all on their way together, and the wait
// for them. In asm, because in front of its own reads the compiler may wait for every load
// into the LDS that is on its way (it cannot know that those go to another buffer), which
// leaves nothing of a pipeline: the first product of the low-rank adapters then took
// 0.97 us a step however many steps were requested ahead.
__device__ __forceinline__ void lds_read(u32x4 (&o)[3], const uint32_t (&at)[3]) {
    asm volatile("ds_read_b128 %0, %3\n\t"
                 "ds_read_b128 %1, %4\n\t"
                 "ds_read_b128 %2, %5\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2])
                 : "v"(at[0]), "v"(at[1]), "v"(at[2])
                 : "memory");
}
__device__ __forceinline__ void lds_read(u32x4 (&o)[4], const uint32_t (&at)[4]) {
    asm volatile("ds_read_b128 %0, %4\n\t"
                 "ds_read_b128 %1, %5\n\t"
                 "ds_read_b128 %2, %6\n\t"
                 "ds_read_b128 %3, %7\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3])
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
                 : "memory");
}
__device__ __forceinline__ void lds_read(u32x4 (&o)[6], const uint32_t (&at)[6]) {
    asm volatile("ds_read_b128 %0, %6\n\t"
                 "ds_read_b128 %1, %7\n\t"
                 "ds_read_b128 %2, %8\n\t"
                 "ds_read_b128 %3, %9\n\t"
                 "ds_read_b128 %4, %10\n\t"
                 "ds_read_b128 %5, %11\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(o[4]), "=&v"(o[5])
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5])
                 : "memory");
}
__device__ __forceinline__ void lds_read(u32x4 (&o)[8], const uint32_t (&at)[8]) {
    asm volatile("ds_read_b128 %0, %8\n\t"
                 "ds_read_b128 %1, %9\n\t"
                 "ds_read_b128 %2, %10\n\t"
                 "ds_read_b128 %3, %11\n\t"
                 "ds_read_b128 %4, %12\n\t"
                 "ds_read_b128 %5, %13\n\t"
                 "ds_read_b128 %6, %14\n\t"
                 "ds_read_b128 %7, %15\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(o[4]), "=&v"(o[5]), "=&v"(o[6]), "=&v"(o[7])
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]), "v"(at[6]), "v"(at[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

}  // namespace moe
