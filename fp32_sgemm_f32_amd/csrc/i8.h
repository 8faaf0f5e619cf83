// The 8-bit integer format and what its kernels share.
//
// A matrix of R rows and K columns: int8 values, rows of kp = K rounded up to
// 128 bytes with zeros beyond K, and fp32 scales, one for a row or one for each
// 128 columns of a row.  So every row starts on a 128-byte line and no product
// masks K.
#pragma once

#include "mx4.h"

namespace sgemm {

inline __host__ __device__ int64_t i8_ld(int64_t cols) { return (cols + 127) / 128 * 128; }

constexpr float kI8Levels = 127.0f;      // the largest whole number of 8 bits
constexpr float kI8Levels16 = 32639.0f;  // of two pieces: 127 * 256 + 127

// A magnitude's bits, as they order: NaN > infinity > finite.
__device__ __forceinline__ uint32_t i8_magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t i8_max(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The scale of a row whose largest magnitude has these bits; NaN where the row
// holds an infinity or NaN.
__device__ __forceinline__ float i8_scale(uint32_t m, float levels) {
    if (m >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    return fmaxf(__fdiv_rn(__uint_as_float(m), levels), 0x1p-126f);
}

// The whole number nearest to v / s, exactly (of two the even one), with inv =
// 1 / s.  v * inv is within 2^-22 of the quotient, relatively, so its nearest
// whole number q is right, or one off where the quotient lies next to a border;
// v - q s, exact in a fused product (its bits lie between the last of s or v and
// s / 2), says on which side.  NaN scales give 0.
__device__ __forceinline__ int i8_nearest(float v, float s, float inv) {
    const float q = rintf(v * inv), r = fmaf(-q, s, v);
    int n = (int)q;
    const float twice = 2.0f * fabsf(r);
    if (twice > s || (twice == s && (n & 1))) n += r > 0.0f ? 1 : -1;
    return s == s ? n : 0;
}

// The largest of the 16 lanes of a row of lanes, in all of them.
__device__ __forceinline__ uint32_t i8_max16(uint32_t m) {
    m = i8_max(m, __builtin_amdgcn_mov_dpp((int)m, 0xB1, 15, 15, true));    // lane ^ 1
    m = i8_max(m, __builtin_amdgcn_mov_dpp((int)m, 0x4E, 15, 15, true));    // lane ^ 2
    m = i8_max(m, __builtin_amdgcn_mov_dpp((int)m, 0x141, 15, 15, true));   // mirrored in eight lanes
    return i8_max(m, __builtin_amdgcn_mov_dpp((int)m, 0x140, 15, 15, true));   // mirrored in sixteen
}

__device__ __forceinline__ uint32_t i8_max8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = i8_max(m, i8_magnitude(v[i]));
    return m;
}

// Eight values as whole numbers, bytes in order.
__device__ __forceinline__ uint2 i8_nearest8(const float (&v)[8], float s, float inv) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4] |= ((uint32_t)i8_nearest(v[i], s, inv) & 255u) << (8 * (i % 4));
    return uint2{w[0], w[1]};
}
// And back.
__device__ __forceinline__ void i8_values8(uint2 q, float s, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)((i < 4 ? q.x : q.y) >> (8 * (i % 4))) * s;
}

// Eight adjacent values of a row from column c on, those before `cols`.
template <int TYPE>
__device__ __forceinline__ void i8_store8(typename MxType<TYPE>::T *row, int c, int cols, const float (&v)[8]) {
    if (c + 8 <= cols) {
        if constexpr (TYPE == SGEMM_TYPE_F32) {
            ((f32v4_any *)(row + c))[0] = f32v4_any{v[0], v[1], v[2], v[3]};
            ((f32v4_any *)(row + c))[1] = f32v4_any{v[4], v[5], v[6], v[7]};
        } else {
            u32v4_any w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)MxType<TYPE>::from(v[2 * i]) | (uint32_t)MxType<TYPE>::from(v[2 * i + 1]) << 16;
            *(u32v4_any *)(row + c) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = MxType<TYPE>::from(v[i]);
    }
}

// Row and eight columns of a thread where a grid of workgroups of `threads`
// goes along rows of `chunks` eights, one row after another.
struct I8Place {
    int64_t row;
    int c;
};
__device__ __forceinline__ I8Place i8_place(int chunks, int threads) {
    const int64_t first = (int64_t)blockIdx.x * threads, row = first / chunks;   // the same for all lanes
    const uint32_t at = (uint32_t)(first - row * chunks) + threadIdx.x, more = at / (uint32_t)chunks;
    return {row + more, (int)(at - more * (uint32_t)chunks) * 8};
}
inline unsigned i8_grid(int64_t rows, int64_t chunks, int threads) { return (unsigned)((rows * chunks + threads - 1) / threads); }

// ---- host: one job per launcher ----

// Rows of a float matrix, by row (q, s).  fold: each column times fold[column]
// first, rounded.
struct I8RowsJob {
    const void *x;
    int64_t ldx;
    int rows, cols, type;
    const float *fold;
    int8_t *q;
    float *s;
};
// Columns of a rows x cols float matrix: q (pieces = 1: cols rows; 2: see
// i8_quant.hip) of `rows` bytes, padded.  fold: each row times fold[row] first.
// part: scratch memory, i8_part_bytes(rows, cols).
struct I8ColsJob {
    const void *x;
    int64_t ldx;
    int rows, cols, type, pieces;
    const float *fold;
    uint32_t *part;
    int8_t *q;
    float *s;
};
// By 128 columns of a row, and both formats back.
struct I8GroupsJob {
    const void *x;
    int64_t ldx;
    int rows, cols, type;
    int8_t *q;
    float *s;
};
struct I8BackJob {
    const int8_t *q;
    const float *s;
    int rows, cols, group, type;
    void *y;
    int64_t ldy;
};
// C (M x N) = alpha A B^T + beta C.  A: M rows of ld(K) bytes, scales sa.  B: N
// rows of ld(K) bytes, scales sb; or with `down` K rows of ld(N) bytes, no
// scales.  pieces = 2 (with down): A holds 16-bit whole numbers in two rows each
// (see i8_quant.hip).
struct I8GemmJob {
    const int8_t *a;
    const float *sa;
    const int8_t *b;
    const float *sb;
    int M, N, K, type, down, pieces;
    float alpha, beta;
    void *c;
    int64_t ldc;
};
struct I8SwigluJob {
    const void *x;        // forward: GU; backward: dH
    int64_t ldx;
    int rows, inner, type;
    int8_t *gq;
    float *gs;
    int8_t *uq;
    float *us;
    void *y;              // forward: H; backward: dGU
    int64_t ldy;
};

// Rows of the matrix that holds 16-bit numbers of n columns in two pieces.
inline __host__ __device__ int64_t i8_piece_rows(int64_t n) { return (n + 31) / 32 * 64; }
int64_t i8_part_bytes(int rows, int cols);

hipError_t launch_i8_rows(const I8RowsJob &j, hipStream_t s);
// Two matrices of one type, in one launch.
hipError_t launch_i8_rows_two(const I8RowsJob &j, const I8RowsJob &k, hipStream_t s);
hipError_t launch_i8_cols(const I8ColsJob &j, hipStream_t s);
hipError_t launch_i8_groups(const I8GroupsJob &j, hipStream_t s);
hipError_t launch_i8_back(const I8BackJob &j, hipStream_t s);
hipError_t launch_i8_gemm(const I8GemmJob &j, int num_cus, hipStream_t s);
hipError_t launch_i8_swiglu_forward(const I8SwigluJob &j, hipStream_t s);
hipError_t launch_i8_swiglu_backward(const I8SwigluJob &j, hipStream_t s);

}  // namespace sgemm
