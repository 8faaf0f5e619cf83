// Quantisation to the microscaled 4-bit format, along the rows, along the
// columns, or both in one pass, and back.
//
// For a block of 32 values with largest magnitude m: the scale byte is
// s = floor(log2 m) - 2 + 127 (held at 0), or, with `noclip`, one more where
// m / 2^(s - 127) would exceed 6, the largest code; each value divided by the
// scale is rounded to the nearest code, ties to the even one, and held at 6.
// A block that holds a NaN or an infinity gets the NaN scale (255) and zero
// codes: the format has neither, and a product must not hide them.
// m is taken on the bits below the sign, where NaN > infinity > finite, so
// one integer maximum finds both; the rounding is the conversion
// instruction's (checked against the definition at every code border and for
// every scale byte).
//
// Bound by HBM: 4 (2) bytes read and 0.53 written per value and direction.
#include "mx4.h"

namespace sgemm {
namespace {

// Lane l's value of lane l ^ 1, l ^ 2 (within four lanes).
__device__ __forceinline__ uint32_t quad_xor1(uint32_t v) { return __builtin_amdgcn_mov_dpp((int)v, 0xB1, 15, 15, true); }
__device__ __forceinline__ uint32_t quad_xor2(uint32_t v) { return __builtin_amdgcn_mov_dpp((int)v, 0x4E, 15, 15, true); }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t max_bits8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// Scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t m, int noclip) {
    const uint32_t e = m >> 23;
    if (e == 255) return 255;
    uint32_t s = e >= 2 ? e - 2 : 0;
    if (noclip && e >= 2 && (m & 0x7fffffu) > 0x400000u) ++s;
    return s;
}

// Codes of eight values under scale byte s, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], uint32_t s) {
    if (s == 255) return 0;
    const float scale = __uint_as_float(s << 23);   // the instruction takes the exponent field: 0 is 2^-127
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
    return c;
}

// Along the rows.  A lane holds 8 adjacent values, four lanes a block, a wave
// 2 rows x 256 columns (full lines both ways), a workgroup 8 rows x 256
// columns.  Rows up to the padding's end get zero scales.
template <int TYPE>
__global__ __launch_bounds__(256) void quant_rows_kernel(MxQuantJob j, int vec) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r = (int64_t)blockIdx.x * 8 + wave * 2 + (lane >> 5);
    const int c = blockIdx.y * 256 + (lane & 31) * 8;
    const int slab = c / kMxSlab, slabs = mx_slabs(j.cols);
    float v[8];
    const bool real = r < j.rows;
    const auto *row = (const typename MxType<TYPE>::T *)j.x + (real ? r : 0) * j.ldx;
    mx_load_edge8<TYPE>(row, c, real ? j.cols : 0, vec, v);
    uint32_t m = max_bits8(v);
    m = umax(m, quad_xor1(m));
    m = umax(m, quad_xor2(m));
    const uint32_t s = scale_byte(m, j.noclip);
    const uint32_t code = codes8(v, s);
    // The word of a slab's four blocks, from lanes 0, 4, 8, 12 of its 16.
    uint32_t word = s << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor(word, 4, 64);
    word |= __shfl_xor(word, 8, 64);
    if (slab >= slabs) return;
    if (real) ((uint32_t *)j.codes)[r * (16 * (int64_t)slabs) + c / 8] = code;
    if ((lane & 15) == 0) ((uint32_t *)j.scales)[slab * mx_plane_rows(j.rows) + r] = word;
}

// Along the columns, or both: a workgroup takes 128 x 128 values.  They are
// read once along the rows (and quantised that way if wanted), laid in LDS as
// they came, and read back down the columns: a thread takes 32 rows of one
// column, a block.  Both ways write whole 64-byte slabs.
template <int TYPE, bool ROWS>
__global__ __launch_bounds__(512) void quant_tile_kernel(MxQuantJob j, int vec) {
    typedef typename MxType<TYPE>::T T;
    __shared__ __attribute__((aligned(16))) T tile[128 * 128];
    __shared__ uint32_t words[128];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t r0 = (int64_t)blockIdx.y * 128;
    const int c0 = blockIdx.x * 128;
    if (tid < 128) words[tid] = 0;
    const int slabs = mx_slabs(j.cols), slabs_t = mx_slabs(j.rows);
    const int lr = tid >> 4, lc = (tid & 15) * 8;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 32 * i + lr;
        const bool real = r < j.rows;
        const T *row = (const T *)j.x + (real ? r : 0) * j.ldx;
        mx_load_edge8<TYPE>(row, c0 + lc, real ? j.cols : 0, vec, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // Rounding back to T is exact: the floats came from it.
        mx_store8<TYPE>(tile + (32 * i + lr) * 128 + lc, v[i]);
        if constexpr (ROWS) {
            const int64_t r = r0 + 32 * i + lr;
            uint32_t m = max_bits8(v[i]);
            m = umax(m, quad_xor1(m));
            m = umax(m, quad_xor2(m));
            const uint32_t s = scale_byte(m, j.noclip);
            const uint32_t code = codes8(v[i], s);
            uint32_t word = s << (8 * ((lane >> 2) & 3));
            word |= __shfl_xor(word, 4, 64);
            word |= __shfl_xor(word, 8, 64);
            if (r < j.rows) ((uint32_t *)j.codes)[r * (16 * (int64_t)slabs) + (c0 + lc) / 8] = code;
            if ((lane & 15) == 0 && r < mx_plane_rows(j.rows))
                ((uint32_t *)j.scales)[blockIdx.x * mx_plane_rows(j.rows) + r] = word;
        }
    }
    __syncthreads();
    const int c = tid & 127, b = tid >> 7;
    float x[4][8];
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[g][i] = MxType<TYPE>::load(tile + (32 * b + 8 * g + i) * 128 + c);
        m = umax(m, max_bits8(x[g]));
    }
    const uint32_t s = scale_byte(m, j.noclip);
    atomicOr(&words[c], s << (8 * b));   // four different bytes: any order gives the same word
    const uint4 code{codes8(x[0], s), codes8(x[1], s), codes8(x[2], s), codes8(x[3], s)};
    if (c0 + c < j.cols) *(uint4 *)(j.codes_t + (c0 + c) * (64 * (int64_t)slabs_t) + blockIdx.y * 64 + b * 16) = code;
    __syncthreads();
    if (tid < 128 && c0 + tid < mx_plane_rows(j.cols))
        ((uint32_t *)j.scales_t)[blockIdx.y * mx_plane_rows(j.cols) + c0 + tid] = words[tid];
}

// Back to floats: a lane takes 8 values, as in quant_rows_kernel.
template <int TYPE>
__global__ __launch_bounds__(256) void dequant_kernel(MxDequantJob j, int vec) {
    typedef typename MxType<TYPE>::T T;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r = (int64_t)blockIdx.x * 8 + wave * 2 + (lane >> 5);
    const int c = blockIdx.y * 256 + (lane & 31) * 8;
    if (r >= j.rows || c >= j.cols) return;
    const int slabs = mx_slabs(j.cols);
    const uint32_t code = ((const uint32_t *)j.codes)[r * (16 * (int64_t)slabs) + c / 8];
    const uint32_t s = j.scales[((c / kMxSlab) * mx_plane_rows(j.rows) + r) * 4 + (c >> 5 & 3)];
    const float scale = __uint_as_float(s << 23);   // 0: 2^-127; 255: NaN
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        auto p = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, scale, 0)
                 : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, scale, 1)
                 : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, scale, 2)
                          : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, scale, 3);
        v[2 * i] = p[0];
        v[2 * i + 1] = p[1];
    }
    T *row = (T *)j.y + r * j.ldy;
    if (vec && c + 8 <= j.cols) {
        mx_store8<TYPE>(row + c, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < j.cols) row[c + i] = MxType<TYPE>::from(v[i]);
}

// Rows start on 16-byte boundaries.
bool vec_rows(const void *p, int64_t ld, int type) {
    const int64_t bytes = type == SGEMM_TYPE_F32 ? 4 : 2;
    return ((uintptr_t)p & 15) == 0 && (ld * bytes & 15) == 0;
}

template <int TYPE>
hipError_t launch_quant(const MxQuantJob &job, hipStream_t s) {
    MxQuantJob j = job;
    int vec = vec_rows(j.x, j.ldx, TYPE);
    void *params[] = {&j, &vec};
    if (!j.codes_t)
        return hipLaunchKernel((const void *)quant_rows_kernel<TYPE>,
                               dim3((unsigned)(mx_plane_rows(j.rows) / 8), (unsigned)((j.cols + 255) / 256)), dim3(256),
                               params, 0, s);
    const dim3 grid((unsigned)mx_slabs(j.cols), (unsigned)mx_slabs(j.rows));
    const void *k = j.codes ? (const void *)quant_tile_kernel<TYPE, true> : (const void *)quant_tile_kernel<TYPE, false>;
    return hipLaunchKernel(k, grid, dim3(512), params, 0, s);
}

template <int TYPE>
hipError_t launch_dequant(const MxDequantJob &job, hipStream_t s) {
    MxDequantJob j = job;
    int vec = vec_rows(j.y, j.ldy, TYPE);
    void *params[] = {&j, &vec};
    return hipLaunchKernel((const void *)dequant_kernel<TYPE>,
                           dim3((unsigned)(((int64_t)j.rows + 7) / 8), (unsigned)((j.cols + 255) / 256)), dim3(256), params,
                           0, s);
}

}  // namespace

hipError_t launch_mx4_quantize(const MxQuantJob &j, hipStream_t s) {
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_quant<SGEMM_TYPE_F32>(j, s);
    case SGEMM_TYPE_BF16: return launch_quant<SGEMM_TYPE_BF16>(j, s);
    case SGEMM_TYPE_F16: return launch_quant<SGEMM_TYPE_F16>(j, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_mx4_dequantize(const MxDequantJob &j, hipStream_t s) {
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_dequant<SGEMM_TYPE_F32>(j, s);
    case SGEMM_TYPE_BF16: return launch_dequant<SGEMM_TYPE_BF16>(j, s);
    case SGEMM_TYPE_F16: return launch_dequant<SGEMM_TYPE_F16>(j, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace sgemm
