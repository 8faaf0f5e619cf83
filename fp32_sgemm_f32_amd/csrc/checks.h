// Argument checks that the files with C entry points share.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <atomic>

#include "abi.h"
#include "sgemm_f32.h"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace sgemm {

inline int type_bytes(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }
inline bool known_type(int type) { return type >= SGEMM_TYPE_F32 && type <= SGEMM_TYPE_F16; }

// One array of a call, in the order of the checks.
struct Span {
    const void *p;
    int64_t bytes;
    int align;
    bool out;
};

inline Span floats(const void *p, int64_t rows, int64_t cols, int64_t ld, int type, bool out) {
    return Span{p, rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * type_bytes(type) : 0, type_bytes(type), out};
}

// Null, alignment, overlap with an output, and device memory, of all arrays
// that hold anything.
template <int N>
int check_spans(const Span (&s)[N], int *dev) {
    for (const Span &x : s)
        if (x.bytes > 0 && !x.p) return SGEMM_ERR_NULL;
    for (const Span &x : s)
        if (x.bytes > 0 && ((uintptr_t)x.p & (x.align - 1))) return SGEMM_ERR_ALIGN;
    for (int i = 0; i < N; ++i)
        for (int k = 0; k < N; ++k) {
            if (i == k || !s[i].out || s[i].bytes <= 0 || s[k].bytes <= 0) continue;
            const uintptr_t a = (uintptr_t)s[i].p, b = (uintptr_t)s[k].p;
            if (a < b + (uint64_t)s[k].bytes && b < a + (uint64_t)s[i].bytes) return SGEMM_ERR_ALIAS;
        }
    const hipError_t e = hipGetDevice(dev);
    if (e != hipSuccess) return hip_fail(e);
    // An array inside an allocation that an earlier one of this call lies in
    // needs no question to the runtime (half a microsecond each).
    uintptr_t lo[N], hi[N];
    int known = 0;
    for (const Span &x : s) {
        if (x.bytes <= 0) continue;
        const uintptr_t p = (uintptr_t)x.p;
        bool inside = false;
        for (int i = 0; i < known && !inside; ++i) inside = p >= lo[i] && p < hi[i] && (uint64_t)x.bytes <= hi[i] - p;
        if (inside) continue;
        const int st = check_device_range(x.p, x.bytes, *dev, &lo[known], &hi[known]);
        if (st != SGEMM_OK) return st;
        ++known;
    }
    return SGEMM_OK;
}

inline int done(hipError_t e) { return e == hipSuccess ? SGEMM_OK : hip_fail(e); }

// Compute units of a device, asked for once.
inline int compute_units(int dev, int *out) {
    static std::atomic<int> known[64];
    if (dev >= 0 && dev < 64 && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return SGEMM_OK;
    const hipError_t e = hipDeviceGetAttribute(out, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return hip_fail(e);
    if (dev >= 0 && dev < 64) known[dev].store(*out, std::memory_order_relaxed);
    return SGEMM_OK;
}

}  // namespace sgemm
