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
// Bound by HBM: 4 (2) bytes read and 0.53 written per value and direction.  8191
// x 16388 floats: along the rows 109 us (5.6 TB/s), both ways 143 (4.7); 8192 x
// 4096 bf16: 14.6 (5.8) and 23.7 (4.3).
#include "mx4.h"

namespace sgemm {
namespace {

constexpr int kDequantLanes = 512;   // of a workgroup of the way back

// Eight values rounded to a 16-bit type.
template <int TYPE>
__device__ __forceinline__ u32v4_any pack8(const float (&v)[8]) {
    u32v4_any w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)MxType<TYPE>::from(v[2 * i]) | (uint32_t)MxType<TYPE>::from(v[2 * i + 1]) << 16;
    return w;
}

// Eight values into LDS, 16-byte aligned.
template <int TYPE>
__device__ __forceinline__ void store8(typename MxType<TYPE>::T *p, const float (&v)[8]) {
    if constexpr (TYPE == SGEMM_TYPE_F32) {
        ((f32v4 *)p)[0] = f32v4{v[0], v[1], v[2], v[3]};
        ((f32v4 *)p)[1] = f32v4{v[4], v[5], v[6], v[7]};
    } else {
        *(uint4 *)p = __builtin_bit_cast(uint4, pack8<TYPE>(v));
    }
}

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
// columns, and workgroups go along a row first (8191 x 16388 floats: 109 us,
// down the rows first 126).  Rows up to the padding's end get zero scales.
template <int TYPE>
__global__ __launch_bounds__(256) void quant_rows_kernel(MxQuantJob j) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 8 + wave * 2 + (lane >> 5);
    const int c = blockIdx.x * 256 + (lane & 31) * 8;
    const int slab = c / kMxSlab, slabs = mx_slabs(j.cols);
    float v[8];
    const bool real = r < j.rows;
    const auto *row = (const typename MxType<TYPE>::T *)j.x + (real ? r : 0) * j.ldx;
    mx_load_edge8<TYPE>(row, c, real ? j.cols : 0, v);
    uint32_t m = max_bits8(v);
    m = umax(m, quad_xor1(m));
    m = umax(m, quad_xor2(m));
    const uint32_t s = scale_byte(m, j.noclip);
    const uint32_t code = codes8(v, s);
    // The word of a slab's four blocks, from lanes 0, 4, 8, 12 of its 16.
    uint32_t word = s << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor(word, 4, 64);
    word |= __shfl_xor(word, 8, 64);
    if (slab >= slabs || r >= mx_plane_rows(j.rows)) return;
    if (real) ((uint32_t *)j.codes)[r * (16 * (int64_t)slabs) + c / 8] = code;
    if ((lane & 15) == 0) ((uint32_t *)j.scales)[slab * mx_plane_rows(j.rows) + r] = word;
}

// Along the columns, or both: a workgroup takes 128 x 128 values.  They are
// read once along the rows (and quantised that way if wanted), laid in LDS as
// they came, and read back down the columns: a thread takes 32 rows of one
// column, a block.  Both ways write whole 64-byte slabs.  One launch serves up
// to two matrices: the first `tiles0` workgroups take tiles of `j0`.
template <int TYPE, bool ROWS>
__global__ __launch_bounds__(512) void quant_tile_kernel(MxQuantJob j0, MxQuantJob j1, int64_t tiles0) {
    const bool one = blockIdx.x >= tiles0;
    const MxQuantJob &j = one ? j1 : j0;
    const int block = (int)(one ? blockIdx.x - tiles0 : blockIdx.x);
    const int bx = block % mx_slabs(j.cols), by = block / mx_slabs(j.cols);
    typedef typename MxType<TYPE>::T T;
    __shared__ __attribute__((aligned(16))) T tile[128 * 128 + 3 * 16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t r0 = (int64_t)by * 128;
    const int c0 = bx * 128;
    const int slabs = mx_slabs(j.cols), slabs_t = mx_slabs(j.rows);
    const int lr = tid >> 4, lc = (tid & 15) * 8;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 32 * i + lr;
        const bool real = r < j.rows;
        const T *row = (const T *)j.x + (real ? r : 0) * j.ldx;
        mx_load_edge8<TYPE>(row, c0 + lc, real ? j.cols : 0, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // Rounding back to T is exact: the floats came from it.
        store8<TYPE>(tile + (32 * i + lr) * 128 + 16 * i + lc, v[i]);
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
                ((uint32_t *)j.scales)[bx * mx_plane_rows(j.rows) + r] = word;
        }
    }
    __syncthreads();
    // Four lanes take the four blocks of a column: their codes are one run of
    // 64 bytes (16 bytes to a row in every store: 25.1 us for both ways of
    // 8192 x 4096 bf16).  The blocks of a column lie 32 rows apart, so every 32
    // rows of the tile are shifted by 16 values to other banks.
    const int c = 16 * (tid >> 6) + (lane >> 2), b = lane & 3;
    float x[4][8];
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[g][i] = MxType<TYPE>::load(tile + (32 * b + 8 * g + i) * 128 + 16 * b + c);
        m = umax(m, max_bits8(x[g]));
    }
    const uint32_t s = scale_byte(m, j.noclip);
    uint32_t word = s << (8 * b);
    word |= quad_xor1(word);
    word |= quad_xor2(word);
    const uint4 code{codes8(x[0], s), codes8(x[1], s), codes8(x[2], s), codes8(x[3], s)};
    if (c0 + c < j.cols) *(uint4 *)(j.codes_t + (c0 + c) * (64 * (int64_t)slabs_t) + (int64_t)by * 64 + b * 16) = code;
    if (b == 0 && c0 + c < mx_plane_rows(j.cols)) ((uint32_t *)j.scales_t)[by * mx_plane_rows(j.cols) + c0 + c] = word;
}

// Back to floats.  A workgroup takes one run of a row, a lane 16 bytes of it,
// stored past the caches.  Workgroups side by side run on different XCDs, and
// a line that two of them write part of costs memory a read: the fewer, longer
// runs, the better (8191 x 16388 and 16388 x 8191 floats, each called over and
// over: 108 and 99 us, with runs of 1 KiB over 8 rows 143 and 139; a fill of as
// many bytes takes 80.  Behind the quantisation, whose results and input fill the
// caches: 125 and 134).
template <int TYPE>
__global__ __launch_bounds__(kDequantLanes) void dequant_kernel(MxDequantJob j) {
    typedef typename MxType<TYPE>::T T;
    constexpr int V = 16 / sizeof(T);
    const int c = (blockIdx.x * kDequantLanes + threadIdx.x) * V;
    const int64_t r = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (c >= j.cols || r >= j.rows) return;
    const uint8_t *codes = j.codes + r * ((int64_t)mx_slabs(j.cols) * kMxSlabBytes) + c / 2;
    const uint32_t code = V == 4 ? *(const uint16_t *)codes : *(const uint32_t *)codes;
    const uint32_t s = j.scales[((c / kMxSlab) * mx_plane_rows(j.rows) + r) * 4 + (c >> 5 & 3)];
    const float f = __uint_as_float(s << 23);   // 0: 2^-127; 255: NaN
    const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, f, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, f, 1);
    float v[8] = {v0[0], v0[1], v1[0], v1[1]};
    if constexpr (V == 8) {
        const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, f, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, f, 3);
        v[4] = v2[0], v[5] = v2[1], v[6] = v3[0], v[7] = v3[1];
    }
    T *y = (T *)j.y + r * j.ldy + c;
    if (c + V <= j.cols) {
        if constexpr (V == 4) __builtin_nontemporal_store(f32v4_any{v[0], v[1], v[2], v[3]}, (f32v4_any *)y);
        else __builtin_nontemporal_store(pack8<TYPE>(v), (u32v4_any *)y);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (c + k < j.cols) y[k] = MxType<TYPE>::from(v[k]);
    }
}

template <int TYPE>
hipError_t launch_quant(const MxQuantJob &job, const MxQuantJob *second, hipStream_t s) {
    MxQuantJob j = job, k = second ? *second : job;
    if (!j.codes_t) {
        void *params[] = {&j};
        const unsigned groups = (unsigned)(mx_plane_rows(j.rows) / 8), y = groups < 32768 ? groups : 32768;
        return hipLaunchKernel((const void *)quant_rows_kernel<TYPE>,
                               dim3((unsigned)((j.cols + 255) / 256), y, (groups + y - 1) / y), dim3(256), params, 0, s);
    }
    int64_t tiles = (int64_t)mx_slabs(j.cols) * mx_slabs(j.rows);
    const int64_t more = second ? (int64_t)mx_slabs(k.cols) * mx_slabs(k.rows) : 0;
    void *params[] = {&j, &k, &tiles};
    const void *f = j.codes ? (const void *)quant_tile_kernel<TYPE, true> : (const void *)quant_tile_kernel<TYPE, false>;
    return hipLaunchKernel(f, dim3((unsigned)(tiles + more)), dim3(512), params, 0, s);
}

template <int TYPE>
hipError_t launch_dequant(const MxDequantJob &job, hipStream_t s) {
    MxDequantJob j = job;
    void *params[] = {&j};
    constexpr int kCols = kDequantLanes * 16 / sizeof(typename MxType<TYPE>::T);
    const unsigned y = j.rows < 32768 ? j.rows : 32768;
    return hipLaunchKernel((const void *)dequant_kernel<TYPE>,
                           dim3((unsigned)((j.cols + kCols - 1) / kCols), y, (j.rows + y - 1) / y), dim3(kDequantLanes), params, 0, s);
}

}  // namespace

hipError_t launch_mx4_quantize(const MxQuantJob &j, hipStream_t s) {
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_quant<SGEMM_TYPE_F32>(j, nullptr, s);
    case SGEMM_TYPE_BF16: return launch_quant<SGEMM_TYPE_BF16>(j, nullptr, s);
    case SGEMM_TYPE_F16: return launch_quant<SGEMM_TYPE_F16>(j, nullptr, s);
    default: return hipErrorInvalidValue;
    }
}

// Two matrices, both ways, in one launch if they are of one type.
hipError_t launch_mx4_quantize_two(const MxQuantJob &j, const MxQuantJob &k, hipStream_t s) {
    if (j.type != k.type) {
        const hipError_t e = launch_mx4_quantize(j, s);
        return e == hipSuccess ? launch_mx4_quantize(k, s) : e;
    }
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_quant<SGEMM_TYPE_F32>(j, &k, s);
    case SGEMM_TYPE_BF16: return launch_quant<SGEMM_TYPE_BF16>(j, &k, s);
    case SGEMM_TYPE_F16: return launch_quant<SGEMM_TYPE_F16>(j, &k, s);
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
