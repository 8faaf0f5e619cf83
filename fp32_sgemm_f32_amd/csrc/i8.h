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

// The whole number n nearest to v / s (of two the even one), as the bits of 1.5
// 2^23 + n: its low bytes are n's.  With inv = 1 / s, v * inv lies within 2^-23 of
// the quotient, relatively, so n is right but where the quotient lies next to a
// border; v - n s, exact in a fused product (its bits lie between the last of s
// or v and s / 2), reaches s / 2 there, and only there is n looked at again.
constexpr float kI8Bias = 12582912.0f;
__device__ __forceinline__ uint32_t i8_bits(float v, float s, float inv, float &rest) {
    const float b = fmaf(v, inv, kI8Bias);
    rest = fabsf(fmaf(-(b - kI8Bias), s, v));
    return __float_as_uint(b);
}
__device__ __forceinline__ uint32_t i8_bits_at_border(float v, float s, float inv) {
    const float b = fmaf(v, inv, kI8Bias), r = fmaf(-(b - kI8Bias), s, v), twice = 2.0f * fabsf(r);
    uint32_t n = __float_as_uint(b);
    if (twice > s || (twice == s && (n & 1))) n += r > 0.0f ? 1 : -1;
    return n;
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

// Eight values as whole numbers, bytes in order; zeros under a NaN scale.
__device__ __forceinline__ uint2 i8_nearest8(const float (&v)[8], float s, float inv) {
    uint32_t n[8];
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float rest;
        n[i] = i8_bits(v[i], s, inv, rest);
        most = fmaxf(most, rest);
    }
    if (__builtin_expect(2.0f * most >= s, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = i8_bits_at_border(v[i], s, inv);
    }
    uint2 w;
    w.x = __builtin_amdgcn_perm(__builtin_amdgcn_perm(n[3], n[2], 0x0c0c0400), __builtin_amdgcn_perm(n[1], n[0], 0x0c0c0400), 0x05040100);
    w.y = __builtin_amdgcn_perm(__builtin_amdgcn_perm(n[7], n[6], 0x0c0c0400), __builtin_amdgcn_perm(n[5], n[4], 0x0c0c0400), 0x05040100);
    return s == s ? w : uint2{0, 0};
}
// And back.
__device__ __forceinline__ void i8_values8(uint2 q, float s, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)((i < 4 ? q.x : q.y) >> (8 * (i % 4))) * s;
}

// Eight adjacent values of a row as they come from memory.
template <int TYPE>
struct I8Raw {
    typedef typename MxType<TYPE>::T E;
    u32v4_any w[TYPE == SGEMM_TYPE_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const E *p) {
        w[0] = ((const u32v4_any *)p)[0];
        if constexpr (TYPE == SGEMM_TYPE_F32) w[1] = ((const u32v4_any *)p)[1];
    }
    // The first n < 8 of them, zeros behind.
    __device__ __forceinline__ void load(const E *p, int n) {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? (TYPE == SGEMM_TYPE_F32 ? ((const uint32_t *)p)[i] : (uint32_t)((const uint16_t *)p)[i]) : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if constexpr (TYPE == SGEMM_TYPE_F32) w[i / 4][i % 4] = v[i];
            else w[0][i / 2] = i % 2 ? w[0][i / 2] | v[i] << 16 : v[i];
    }
    __device__ __forceinline__ void clear() {
        w[0] = u32v4_any{0, 0, 0, 0};
        if constexpr (TYPE == SGEMM_TYPE_F32) w[1] = w[0];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if constexpr (TYPE == SGEMM_TYPE_F32) {
                v[i] = __uint_as_float(w[i / 4][i % 4]);
            } else {
                const uint16_t h = (uint16_t)(w[0][i / 2] >> (16 * (i % 2)));
                v[i] = MxType<TYPE>::load(&h);
            }
    }
};

// N eights of a row, from columns c, c + step, ... on; zeros at and after
// `cols`.  All loads are in flight before any is waited for.
template <int TYPE, int N>
__device__ __forceinline__ void i8_load_row(const typename MxType<TYPE>::T *row, int c, int step, int cols, I8Raw<TYPE> (&r)[N]) {
    const int whole = cols & ~7;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        r[i].clear();
        if (c + i * step < whole) r[i].load(row + c + i * step);
    }
    if (whole < cols) {   // one lane's
        I8Raw<TYPE> last;
        last.load(row + whole, cols - whole);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i * step == whole) r[i] = last;
    }
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

// A sum times its row's and its column's scale: the smaller first, which
// neither overflows nor underflows where the result does not.
__device__ __forceinline__ float i8_scaled(float sum, float x, float y) {
    const bool less = x < y;   // (where one is NaN, it comes second)
    return sum * (less ? x : y) * (less ? y : x);
}

// ---- host: one job per launcher ----

// Rows of a float matrix, by row (q, s).
struct I8RowsJob {
    const void *x;
    int64_t ldx;
    int rows, cols, type;
    int8_t *q;
    float *s;
};
// Columns of a rows x cols float matrix, as rows of `rows` bytes, padded.  fold:
// each row times fold[row] first.  part: scratch memory, i8_part_bytes(rows, cols).
struct I8ColsJob {
    const void *x;
    int64_t ldx;
    int rows, cols, type;
    const float *fold;
    uint32_t *part;
    int8_t *q;
    float *s;
};
// A gradient both ways: times by_col, by row (q, s), and times by_row, by column
// in 16 bits (qt, st; two rows for a column, see i8_quant.hip).  part: scratch
// memory, i8_both_part_bytes(rows, cols).
struct I8BothJob {
    const void *x;
    int64_t ldx;
    int rows, cols, type;
    const float *by_col, *by_row;
    uint32_t *part;
    int8_t *q;
    float *s;
    int8_t *qt;
    float *st;
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
int64_t i8_both_part_bytes(int rows, int cols);

hipError_t launch_i8_rows(const I8RowsJob &j, hipStream_t s);
// Two matrices of one type, in one launch.
hipError_t launch_i8_rows_two(const I8RowsJob &j, const I8RowsJob &k, hipStream_t s);
hipError_t launch_i8_cols(const I8ColsJob &j, hipStream_t s);
hipError_t launch_i8_both(const I8BothJob &j, hipStream_t s);
hipError_t launch_i8_groups(const I8GroupsJob &j, hipStream_t s);
hipError_t launch_i8_back(const I8BackJob &j, hipStream_t s);
hipError_t launch_i8_gemm(const I8GemmJob &j, int num_cus, hipStream_t s);
// Two products, down, the second with pieces = 2 (and a result in fp32).
hipError_t launch_i8_gemm_two(const I8GemmJob &j, const I8GemmJob &k, int num_cus, hipStream_t s);
// The same for at most kI8ThinRows rows of A or B (not down, one piece): weights
// streamed past tokens.  floats: A is quantised on the way (type j.type, leading
// dimension ldx).
constexpr int kI8ThinRows = 8;
bool i8_thin_takes(int M, int N, int K);
bool i8_thin_takes_floats(int M, int N, int K);
hipError_t launch_i8_thin(const I8GemmJob &j, const void *floats, int64_t ldx, int num_cus, hipStream_t s);
hipError_t launch_i8_swiglu_forward(const I8SwigluJob &j, hipStream_t s);
hipError_t launch_i8_swiglu_backward(const I8SwigluJob &j, hipStream_t s);

}  // namespace sgemm
