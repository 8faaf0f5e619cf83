// The microscaled 4-bit format (MXFP4) and what its kernels share.
//
// A matrix of R rows and K columns is held in blocks of 32 values along a
// row: 4-bit codes (sign, then the index into 0, 0.5, 1, 1.5, 2, 3, 4, 6) and
// one scale byte s per block, standing for 2^(s - 127); s = 255 makes the
// block NaN.  Kp = K rounded up to 128 (a slab: four blocks).
//   codes   R rows of Kp / 2 bytes, the even column in the low four bits
//   scales  Kp / 128 planes (one per slab) of Rp = R rounded up to 32 words;
//           byte b of a row's word is the scale of block b of the slab
// Codes beyond K and scales beyond K and R are zeros.  So every row of codes
// starts on a 64-byte boundary, a tile needs no mask along K, and the scales
// of neighbouring rows lie side by side, as the tiles read them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sgemm_f32.h"

namespace sgemm {

constexpr int kMxSlab = 128;      // columns of a slab
constexpr int kMxSlabBytes = 64;  // bytes of its codes in a row

inline __host__ __device__ int mx_slabs(int cols) { return (int)(((int64_t)cols + kMxSlab - 1) / kMxSlab); }
inline __host__ __device__ int64_t mx_plane_rows(int64_t rows) { return (rows + 31) / 32 * 32; }

typedef float f32v4 __attribute__((ext_vector_type(4)));
typedef float f32v16 __attribute__((ext_vector_type(16)));
typedef int i32v4 __attribute__((ext_vector_type(4)));
typedef int i32v8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16v2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));

template <int TYPE>
struct MxType;
template <>
struct MxType<SGEMM_TYPE_F32> {
    typedef float T;
    static __device__ __forceinline__ float load(const T *p) { return *p; }
    static __device__ __forceinline__ T from(float v) { return v; }
};
template <>
struct MxType<SGEMM_TYPE_BF16> {
    typedef uint16_t T;
    static __device__ __forceinline__ float load(const T *p) { return __uint_as_float((uint32_t)*p << 16); }
    // Round to nearest, ties to even (NaN stays NaN).
    static __device__ __forceinline__ T from(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
template <>
struct MxType<SGEMM_TYPE_F16> {
    typedef uint16_t T;
    static __device__ __forceinline__ float load(const T *p) { return (float)__builtin_bit_cast(_Float16, *p); }
    static __device__ __forceinline__ T from(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};

// 16 bytes at any element's address: the hardware takes wide loads and stores
// of global memory at any alignment (a line more where they straddle one), so
// odd leading dimensions and shifted views need no narrow path.
typedef float f32v4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32v4_any __attribute__((ext_vector_type(4), aligned(2)));

// Eight adjacent values as floats.
template <int TYPE>
__device__ __forceinline__ void mx_load8(const typename MxType<TYPE>::T *p, float (&v)[8]) {
    if constexpr (TYPE == SGEMM_TYPE_F32) {
        const f32v4_any a = ((const f32v4_any *)p)[0], b = ((const f32v4_any *)p)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
        const u32v4_any w = *(const u32v4_any *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint16_t lo = (uint16_t)w[i], hi = (uint16_t)(w[i] >> 16);
            v[2 * i] = MxType<TYPE>::load(&lo);
            v[2 * i + 1] = MxType<TYPE>::load(&hi);
        }
    }
}

// Eight values of a row from column c on, zeros at and after `cols`.
template <int TYPE>
__device__ __forceinline__ void mx_load_edge8(const typename MxType<TYPE>::T *row, int c, int cols, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (c + 8 <= cols) {
        mx_load8<TYPE>(row + c, v);
    } else if (c < cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) v[i] = MxType<TYPE>::load(row + c + i);
    }
}

// ---- host: one job per launcher ----

struct MxQuantJob {
    const void *x;
    int64_t ldx;
    int rows, cols, type, noclip;
    uint8_t *codes, *scales;        // along the rows; NULL: not wanted
    uint8_t *codes_t, *scales_t;    // of the transposed matrix; NULL: not wanted
};
struct MxDequantJob {
    const uint8_t *codes, *scales;
    int rows, cols, type;
    void *y;
    int64_t ldy;
};
struct MxGemmJob {
    const uint8_t *a, *sa, *b, *sb;
    int M, N, K, type;
    float alpha, beta;
    void *c;
    int64_t ldc;
};

hipError_t launch_mx4_quantize(const MxQuantJob &j, hipStream_t s);
hipError_t launch_mx4_quantize_two(const MxQuantJob &j, const MxQuantJob &k, hipStream_t s);
hipError_t launch_mx4_dequantize(const MxDequantJob &j, hipStream_t s);
hipError_t launch_mx4_gemm(const MxGemmJob &j, int num_cus, hipStream_t s);
// Two products, the second with a result in fp32; in one launch where both take the same tiles.
hipError_t launch_mx4_gemm_two(const MxGemmJob &j, const MxGemmJob &k, int num_cus, hipStream_t s);

}  // namespace sgemm
