// What the kernels that load tiles straight into LDS share: the loads, the
// buffer resources they go through, the waits, and stores of a few adjacent
// values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace sgemm {

typedef int i32v4 __attribute__((ext_vector_type(4)));

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 (4) bytes per lane from the resource's base + voff into LDS at
// m0 + 16 (4) * lane; lanes out of the resource's range leave zeros.
__device__ __forceinline__ void dma16(i32v4 rsrc, uint32_t voff, uint32_t m0v) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "s"(m0v)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4(i32v4 rsrc, uint32_t voff, uint32_t m0v) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "s"(m0v)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// No instruction moves across.
__device__ __forceinline__ void fence_order() { __builtin_amdgcn_sched_barrier(0); }

// f(0), f(1), ... with compile-time arguments FIRST .. END - 1.
template <int FIRST, int END, class F>
__device__ __forceinline__ void each(F f) {
    if constexpr (FIRST < END) {
        f(std::integral_constant<int, FIRST>{});
        each<FIRST + 1, END>(f);
    }
}

// At most VM of this wave's loads still in flight, its LDS reads done, and
// every wave of the workgroup here.
template <int VM>
__device__ __forceinline__ void meet() {
    static_assert(VM >= 0 && VM < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

__device__ __forceinline__ i32v4 resource(const void *p, int64_t bytes) {
    const uint64_t a = (uint64_t)p;
    return i32v4{(int)(uint32_t)a, (int)(uint32_t)(a >> 32), (int)(uint32_t)(bytes > 0 ? bytes : 0), 0x00020000};
}
__device__ __forceinline__ void advance(i32v4 &r, int64_t bytes) {
    const uint64_t a = (((uint64_t)(uint32_t)r[1] << 32) | (uint32_t)r[0]) + (uint64_t)bytes;
    r[0] = (int)(uint32_t)a;
    r[1] = (int)(uint32_t)(a >> 32);
}

template <int F, class T>
struct __attribute__((packed, aligned(sizeof(T)))) Vec {   // stored at any element's address
    T v[F];
};

// A store, past the caches if PAST.
template <bool PAST, class V>
__device__ __forceinline__ void store(V *p, const V &v) {
    typedef uint32_t u32_any __attribute__((aligned(2)));
    typedef uint32_t u32v2_any __attribute__((ext_vector_type(2), aligned(2)));
    if constexpr (PAST && sizeof(V) == 4) __builtin_nontemporal_store(__builtin_bit_cast(uint32_t, v), (u32_any *)p);
    else if constexpr (PAST && sizeof(V) == 8) __builtin_nontemporal_store(__builtin_bit_cast(u32v2_any, v), (u32v2_any *)p);
    else *p = v;
}

}  // namespace sgemm
