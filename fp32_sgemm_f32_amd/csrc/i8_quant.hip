// Quantisation to 8-bit integers, by rows, by columns (transposed on the way)
// and by groups of 128 columns, and back.
//
// A row's scale follows from its largest magnitude m: s = max(m / 127, 2^-126),
// and x is held as the whole number nearest to x / s.  m is taken on the bits
// below the sign, so that one integer maximum finds NaN and infinities too.
//
// Gradients that go into an integer product are first multiplied by the scales
// that stand along the product's sum (fold).  By columns they are held in 16
// bits: n = 256 h + l with h and l signed bytes, the two rows of a column 32
// apart in a matrix of twice the rows (rows 64 b + i hold h, 64 b + 32 + i l of
// column 32 b + i), which is how a fragment of a matrix instruction takes them.
//
// Bound by HBM (a copy runs at 5.1 TB/s): 8191 x 16388 floats in groups 129 us (5.2
// TB/s), back 113 to 129 (5.2 to 6.0); rows of 12288 x 4096 bf16 29 us (5.2); a
// gradient of 8192 x 4096 bf16 28 us by row with the columns' largest magnitudes
// (3.9), 4 to join those, 27 by column (4.9); any bf16 matrix of that size by
// column 12 for the largest magnitudes (5.5) and 21 to write it (4.8), 16384 x 16384
// 128 (4.2) and 175 (4.6).  Rounding once cost twenty instructions a value and was
// half of a row's time; now it takes five, and looks again only next to a border
// (i8_bits).
#include "i8.h"

namespace sgemm {
namespace {

constexpr int kKeep = 4;   // eights of a row that a lane keeps in registers between the two passes

// WAVES waves take a row, few enough that their lanes keep it between the two
// passes (longer ones are read again); four rows a workgroup where that is one.
// All loads of a lane are out before it waits for any.
template <int TYPE, int WAVES>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void i8_rows_kernel(I8RowsJob j0, I8RowsJob j1, int64_t blocks0) {
    constexpr int T = 64 * WAVES, ROWS = WAVES == 1 ? 4 : 1;
    typedef typename MxType<TYPE>::T E;
    const bool second = blockIdx.x >= blocks0;
    const I8RowsJob &j = second ? j1 : j0;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, t = WAVES == 1 ? lane : (int)threadIdx.x;
    const int64_t row = (blockIdx.x - (second ? blocks0 : 0)) * ROWS + (WAVES == 1 ? wave : 0);
    if (row >= j.rows) return;
    const E *x = (const E *)j.x + row * j.ldx;
    const int ld = (int)i8_ld(j.cols);
    // Values kKeep T eights from c on, and their largest magnitude.
    const auto load = [&](int c, float (&v)[kKeep][8], uint32_t m) {
        I8Raw<TYPE> raw[kKeep];
        i8_load_row<TYPE>(x, c, 8 * T, j.cols, raw);
#pragma unroll
        for (int i = 0; i < kKeep; ++i) raw[i].get(v[i]);
#pragma unroll
        for (int i = 0; i < kKeep; ++i) m = i8_max(m, i8_max8(v[i]));
        return m;
    };
    float v[kKeep][8];
    uint32_t m = load(8 * t, v, 0);
    for (int c = 8 * (t + T * kKeep); c < j.cols; c += 8 * T * kKeep) {
        float w[kKeep][8];
        m = load(c, w, m);
    }
    m = i8_max16(m);
    m = i8_max(m, __shfl_xor(m, 16, 64));
    m = i8_max(m, __shfl_xor(m, 32, 64));
    if constexpr (WAVES > 1) {
        __shared__ uint32_t part[WAVES];
        if (lane == 0) part[wave] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) m = i8_max(m, part[i]);
    }
    const float s = i8_scale(m, kI8Levels), inv = 1.0f / s;
    int8_t *q = j.q + row * ld;
    for (int c0 = 8 * t; c0 < ld; c0 += 8 * T * kKeep) {
        if (c0 > 8 * t) load(c0, v, 0);
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int c = c0 + 8 * T * i;
            if (c < ld) *(uint2 *)(q + c) = i8_nearest8(v[i], s, inv);
        }
    }
    if (t == 0) j.s[row] = s;
}

// ---- by columns ----

constexpr int kMostParts = 64;
inline __host__ __device__ int rows_of_part(int rows) {
    const int per = (rows + kMostParts - 1) / kMostParts;
    return per > 64 ? per : 64;
}
inline __host__ __device__ int parts_of(int rows) { return (rows + rows_of_part(rows) - 1) / rows_of_part(rows); }

// The largest magnitudes of 128 columns in a part of the rows.
template <int TYPE>
__global__ __launch_bounds__(256) void i8_part_kernel(I8ColsJob j) {
    typedef typename MxType<TYPE>::T E;
    __shared__ uint32_t most[16][128];
    const int c = 8 * (threadIdx.x & 15), r = threadIdx.x >> 4, c0 = blockIdx.x * 128;
    const int per = rows_of_part(j.rows), begin = blockIdx.y * per, end = begin + per < j.rows ? begin + per : j.rows;
    uint32_t m[8] = {};
#pragma unroll 4
    for (int row = begin + r; row < end; row += 16) {
        float v[8];
        const E *x = (const E *)j.x + row * j.ldx;
        if (c0 + 128 <= j.cols) mx_load8<TYPE>(x + c0 + c, v);
        else mx_load_edge8<TYPE>(x, c0 + c, j.cols, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = i8_max(m[i], i8_magnitude(v[i]));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) most[r][c + i] = m[i];
    __syncthreads();
    if (threadIdx.x < 128) {
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) all = i8_max(all, most[i][threadIdx.x]);
        j.part[(int64_t)blockIdx.y * i8_ld(j.cols) + c0 + threadIdx.x] = all;
    }
}

// 128 columns x ROWS rows, written as rows.  fold: each row times fold[row]
// first.
template <int TYPE, int PIECES, int ROWS>
__global__ __launch_bounds__(256) void i8_cols_kernel(I8ColsJob j, int parts) {
    typedef typename MxType<TYPE>::T E;
    // The bytes of a column, in quads of four words: quad q at q ^ (column / 8).
    // The 16 columns that a wave writes at a time, whose rows begin at the same
    // bank, so take QUADS different quads: two to a bank with 128 rows, four with
    // 64.  (Conflicts are 61 to 66% of the cycles in which LDS is busy, those a
    // quarter to a third of the kernel's.)
    constexpr int WORDS = ROWS / 4, QUADS = ROWS / 16;
    __shared__ __attribute__((aligned(16))) uint32_t tile[PIECES][128][WORDS];
    const auto word = [](int column, int at) { return (((at >> 2) ^ (column >> 3)) & (QUADS - 1)) * 4 + (at & 3); };
    __shared__ uint32_t most[128];
    __shared__ float scale[128], inverse[128];
    const int tid = threadIdx.x, c0 = blockIdx.x * 128, ld = (int)i8_ld(j.rows);
    {
        const int c = tid & 127;
        uint32_t m = 0;
#pragma unroll 8
        for (int p = tid >> 7; p < parts; p += 2) m = i8_max(m, j.part[p * i8_ld(j.cols) + c0 + c]);
        if (tid < 128) most[c] = m;
        __syncthreads();
        if (tid >= 128) {
            const float s = i8_scale(i8_max(m, most[c]), PIECES == 2 ? kI8Levels16 : kI8Levels);
            scale[c] = s;
            inverse[c] = 1.0f / s;
            if (blockIdx.y == 0 && c0 + c < j.cols) j.s[c0 + c] = s;
        }
        __syncthreads();
    }
    const int c = 8 * (tid & 15);
    const int r0 = blockIdx.y * ROWS;
    {
#pragma unroll
        for (int it = 0; it < ROWS / 64; ++it) {
            const int four = (tid >> 4) + 16 * it;   // four rows, one word of a column
            float v[4][8];
            if (c0 + 128 <= j.cols && r0 + ROWS <= j.rows) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mx_load8<TYPE>((const E *)j.x + (r0 + 4 * four + k) * j.ldx + c0 + c, v[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = r0 + 4 * four + k;
                    const bool real = row < j.rows;
                    mx_load_edge8<TYPE>((const E *)j.x + (real ? row : 0) * j.ldx, c0 + c, real ? j.cols : 0, v[k]);
                }
            }
            if (j.fold)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = r0 + 4 * four + k;
                    const float f = row < j.rows ? j.fold[row] : 1.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[k][i] *= f;
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = scale[c + i], inv = inverse[c + i];
                uint32_t q[4];
                float rests = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float rest;
                    q[k] = i8_bits(v[k][i], s, inv, rest);
                    rests = fmaxf(rests, rest);
                }
                if (__builtin_expect(2.0f * rests >= s, 0)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] = i8_bits_at_border(v[k][i], s, inv);
                }
                if constexpr (PIECES == 2) {
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = q[k] + 128;   // its second byte
                    const uint32_t high = __builtin_amdgcn_perm(__builtin_amdgcn_perm(h[3], h[2], 0x0c0c0501),
                                                                __builtin_amdgcn_perm(h[1], h[0], 0x0c0c0501), 0x05040100);
                    tile[0][c + i][word(c + i, four)] = s == s ? high : 0;
                }
                const uint32_t low = __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[3], q[2], 0x0c0c0400),
                                                           __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400), 0x05040100);
                tile[PIECES - 1][c + i][word(c + i, four)] = s == s ? low : 0;
            }
        }
        __syncthreads();
        for (int i = tid / QUADS; i < PIECES * 128; i += 256 / QUADS) {
            const int piece = i >> 7, n = i & 127, column = c0 + n, quad = tid % QUADS;
            if (column >= j.cols) continue;
            const int64_t row = PIECES == 2 ? (int64_t)(column >> 5) * 64 + piece * 32 + (column & 31) : column;
            *(uint4 *)(j.q + row * ld + r0 + 16 * quad) = *(const uint4 *)&tile[piece][n][word(n, 4 * quad)];
        }
    }
}

// The largest of `per` parts each.
__global__ __launch_bounds__(256) void i8_join_kernel(const uint32_t *part, uint32_t *out, int parts, int per, int ld) {
    const int c = blockIdx.x * 256 + threadIdx.x, first = blockIdx.y * per, end = first + per < parts ? first + per : parts;
    if (c >= ld) return;
    uint32_t m = 0;
#pragma unroll 8
    for (int p = first; p < end; ++p) m = i8_max(m, part[(int64_t)p * ld + c]);
    out[(int64_t)blockIdx.y * ld + c] = m;
}

// ---- a gradient, both ways ----
//
// One pass over dY (where its rows fit): each value times its column's scale,
// by row in 8 bits; and the columns' largest magnitudes of each value times its
// row's scale, over the rows of a workgroup, for i8_cols_kernel.

// Eight rows, so that two workgroups fit on a CU and one reads while the other
// writes (8192 x 4096 bf16: 28 us; sixteen rows and one workgroup 39).
// A workgroup of 512 takes kBothRows rows at a time, each lane eight columns of
// them (or, KEEP = false, of several runs of 4096 columns, read twice).
constexpr int kBothRows = 8;

template <int TYPE, bool KEEP>
__global__ __launch_bounds__(512) void i8_both_kernel(I8BothJob j, int groups) {
    typedef typename MxType<TYPE>::T E;
    constexpr int R = kBothRows;
    __shared__ uint32_t most[8][R];
    __shared__ float scale[R], inverse[R];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int ld = (int)i8_ld(j.cols), runs = KEEP ? 1 : (ld + 4095) / 4096;
    for (int group = blockIdx.x; group < groups; group += gridDim.x) {
        const int r0 = group * R;
        I8Raw<TYPE> raw[R];
        float w[8];
        const auto load = [&](int run) {
            const int c = 4096 * run + 8 * tid;
            mx_load_edge8<SGEMM_TYPE_F32>(j.by_col, c, j.cols, w);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                I8Raw<TYPE> one[1];
                i8_load_row<TYPE>((const E *)j.x + (r0 + r < j.rows ? r0 + r : 0) * j.ldx, c, 0, r0 + r < j.rows ? j.cols : 0, one);
                raw[r] = one[0];
            }
        };
        uint32_t rm[R] = {};
        for (int run = 0; run < runs; ++run) {
            load(run);
            uint32_t cm[8] = {};
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float v[8];
                raw[r].get(v);
                const float f = r0 + r < j.rows ? j.by_row[r0 + r] : 1.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    rm[r] = i8_max(rm[r], i8_magnitude(v[i] * w[i]));
                    cm[i] = i8_max(cm[i], i8_magnitude(v[i] * f));
                }
            }
            const int c = 4096 * run + 8 * tid;
            if (c < ld) {
                uint4 *p = (uint4 *)(j.part + (int64_t)blockIdx.x * ld + c);
                if (group != (int)blockIdx.x) {   // this thread's own, of the rows before
                    const uint4 a = p[0], b = p[1];
                    cm[0] = i8_max(cm[0], a.x), cm[1] = i8_max(cm[1], a.y), cm[2] = i8_max(cm[2], a.z), cm[3] = i8_max(cm[3], a.w);
                    cm[4] = i8_max(cm[4], b.x), cm[5] = i8_max(cm[5], b.y), cm[6] = i8_max(cm[6], b.z), cm[7] = i8_max(cm[7], b.w);
                }
                p[0] = uint4{cm[0], cm[1], cm[2], cm[3]};
                p[1] = uint4{cm[4], cm[5], cm[6], cm[7]};
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t m = i8_max16(rm[r]);
            m = i8_max(m, __shfl_xor(m, 16, 64));
            m = i8_max(m, __shfl_xor(m, 32, 64));
            if (lane == 0) most[wave][r] = m;
        }
        __syncthreads();
        if (tid < R) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = i8_max(m, most[i][tid]);
            const float s = i8_scale(m, kI8Levels);
            scale[tid] = s;
            inverse[tid] = 1.0f / s;
            if (r0 + tid < j.rows) j.s[r0 + tid] = s;
        }
        __syncthreads();
        for (int run = 0; run < runs; ++run) {
            if (!KEEP) load(run);
            const int c = 4096 * run + 8 * tid;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (c < ld && r0 + r < j.rows) {
                    float v[8];
                    raw[r].get(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= w[i];
                    *(uint2 *)(j.q + (int64_t)(r0 + r) * ld + c) = i8_nearest8(v, scale[r], inverse[r]);
                }
        }
        // (the next group writes `most` again only after its loads, and `scale` behind a barrier)
    }
}

// ---- by groups, and back ----

template <int TYPE>
__global__ __launch_bounds__(256) void i8_groups_kernel(I8GroupsJob j) {
    const int chunks = (int)(i8_ld(j.cols) / 8);
    const I8Place at = i8_place(chunks, 256);
    const bool real = at.row < j.rows;
    float v[8];
    mx_load_edge8<TYPE>((const typename MxType<TYPE>::T *)j.x + (real ? at.row : 0) * j.ldx, at.c, real ? j.cols : 0, v);
    const float s = i8_scale(i8_max16(i8_max8(v)), kI8Levels), inv = 1.0f / s;
    if (!real) return;
    *(uint2 *)(j.q + (at.row * chunks) * 8 + at.c) = i8_nearest8(v, s, inv);
    if ((threadIdx.x & 15) == 0) j.s[at.row * (chunks / 16) + at.c / 128] = s;
}

template <int TYPE>
__global__ __launch_bounds__(256) void i8_back_kernel(I8BackJob j) {
    const int chunks = (j.cols + 7) / 8;
    const I8Place at = i8_place(chunks, 256);
    if (at.row >= j.rows) return;
    const int64_t ld = i8_ld(j.cols);
    float v[8];
    i8_values8(*(const uint2 *)(j.q + at.row * ld + at.c), j.s[j.group ? at.row * (ld / 128) + at.c / 128 : at.row], v);
    i8_store8<TYPE>((typename MxType<TYPE>::T *)j.y + at.row * j.ldy, at.c, j.cols, v);
}

// ---- launches ----

template <int TYPE, int WAVES>
hipError_t rows(const I8RowsJob &first, const I8RowsJob &second, hipStream_t s) {
    constexpr int ROWS = WAVES == 1 ? 4 : 1;
    I8RowsJob j = first, k = second;
    int64_t head = ((int64_t)j.rows + ROWS - 1) / ROWS;
    const int64_t all = head + ((int64_t)k.rows + ROWS - 1) / ROWS;
    void *params[] = {&j, &k, &head};
    return hipLaunchKernel((const void *)i8_rows_kernel<TYPE, WAVES>, dim3((unsigned)all), dim3(WAVES == 1 ? 256 : 64 * WAVES), params, 0, s);
}

// Few enough waves that a lane keeps its part of a row.
template <int TYPE>
hipError_t rows_type(const I8RowsJob &j, const I8RowsJob &k, hipStream_t s) {
    const int cols = j.cols > k.cols ? j.cols : k.cols;
    if (cols <= 64 * 8 * kKeep) return rows<TYPE, 1>(j, k, s);
    if (cols <= 256 * 8 * kKeep) return rows<TYPE, 4>(j, k, s);
    return rows<TYPE, 16>(j, k, s);
}

// Tiles of 64 rows, or 128 where there are many.
template <int TYPE, int PIECES>
hipError_t cols_tiles(I8ColsJob j, int parts, hipStream_t s) {
    const int across = (int)(i8_ld(j.cols) / 128), down = (int)(i8_ld(j.rows) / 128);
    const bool many = (int64_t)across * down >= 512;
    void *params[] = {&j, &parts};
    return hipLaunchKernel(many ? (const void *)i8_cols_kernel<TYPE, PIECES, 128> : (const void *)i8_cols_kernel<TYPE, PIECES, 64>,
                           dim3((unsigned)across, (unsigned)(many ? down : 2 * down)), dim3(256), params, 0, s);
}

template <int TYPE>
hipError_t cols_type(const I8ColsJob &job, hipStream_t s) {
    I8ColsJob j = job;
    void *params[] = {&j};
    const hipError_t e = hipLaunchKernel((const void *)i8_part_kernel<TYPE>, dim3((unsigned)(i8_ld(j.cols) / 128), (unsigned)parts_of(j.rows)),
                                         dim3(256), params, 0, s);
    return e == hipSuccess ? cols_tiles<TYPE, 1>(j, parts_of(j.rows), s) : e;
}

// Two workgroups of i8_both_kernel on a CU, each with largest magnitudes of its
// own; where they are many they are joined to kJoined first, in a kernel of 4
// us: every workgroup of i8_cols_kernel reads them all (8192 x 4096: 27 us so,
// 42 with 256 of them and four tiles to a workgroup).
constexpr int kMostBoth = 512, kJoined = 16;
int both_parts(int rows) {
    const int groups = (rows + kBothRows - 1) / kBothRows;
    return groups < kMostBoth ? groups : kMostBoth;
}

template <int TYPE>
hipError_t both_type(I8BothJob j, hipStream_t s) {
    int groups = (j.rows + kBothRows - 1) / kBothRows, parts = both_parts(j.rows), ld = (int)i8_ld(j.cols);
    void *params[] = {&j, &groups};
    hipError_t e = hipLaunchKernel(j.cols <= 4096 ? (const void *)i8_both_kernel<TYPE, true> : (const void *)i8_both_kernel<TYPE, false>,
                                   dim3((unsigned)parts), dim3(512), params, 0, s);
    if (e != hipSuccess) return e;
    uint32_t *part = j.part;
    if (parts > 4 * kJoined) {
        int per = (parts + kJoined - 1) / kJoined;
        part += (int64_t)parts * ld;
        void *join[] = {&j.part, &part, &parts, &per, &ld};
        e = hipLaunchKernel((const void *)i8_join_kernel, dim3((unsigned)((ld + 255) / 256), (unsigned)((parts + per - 1) / per)), dim3(256), join, 0, s);
        if (e != hipSuccess) return e;
        parts = (parts + per - 1) / per;
    }
    return cols_tiles<TYPE, 2>({j.x, j.ldx, j.rows, j.cols, TYPE, j.by_row, part, j.qt, j.st}, parts, s);
}

template <int TYPE>
hipError_t groups_type(const I8GroupsJob &job, hipStream_t s) {
    I8GroupsJob j = job;
    void *params[] = {&j};
    return hipLaunchKernel((const void *)i8_groups_kernel<TYPE>, dim3(i8_grid(j.rows, i8_ld(j.cols) / 8, 256)), dim3(256), params, 0, s);
}

template <int TYPE>
hipError_t back_type(const I8BackJob &job, hipStream_t s) {
    I8BackJob j = job;
    void *params[] = {&j};
    return hipLaunchKernel((const void *)i8_back_kernel<TYPE>, dim3(i8_grid(j.rows, (j.cols + 7) / 8, 256)), dim3(256), params, 0, s);
}

}  // namespace

int64_t i8_part_bytes(int rows, int cols) { return rows > 0 ? parts_of(rows) * i8_ld(cols) * 4 : 0; }
int64_t i8_both_part_bytes(int rows, int cols) { return (int64_t)(both_parts(rows) + kJoined) * i8_ld(cols) * 4; }

#define I8_BY_TYPE(type, call)                          \
    switch (type) {                                     \
    case SGEMM_TYPE_F32: return call(SGEMM_TYPE_F32);   \
    case SGEMM_TYPE_BF16: return call(SGEMM_TYPE_BF16); \
    case SGEMM_TYPE_F16: return call(SGEMM_TYPE_F16);   \
    default: return hipErrorInvalidValue;               \
    }

hipError_t launch_i8_rows_two(const I8RowsJob &j, const I8RowsJob &k, hipStream_t s) {
#define CALL(T) rows_type<T>(j, k, s)
    I8_BY_TYPE(j.type, CALL)
#undef CALL
}

hipError_t launch_i8_rows(const I8RowsJob &j, hipStream_t s) {
    I8RowsJob none = j;
    none.rows = 0;
    return launch_i8_rows_two(j, none, s);
}

hipError_t launch_i8_cols(const I8ColsJob &j, hipStream_t s) {
#define CALL(T) cols_type<T>(j, s)
    I8_BY_TYPE(j.type, CALL)
#undef CALL
}

hipError_t launch_i8_both(const I8BothJob &j, hipStream_t s) {
#define CALL(T) both_type<T>(j, s)
    I8_BY_TYPE(j.type, CALL)
#undef CALL
}

hipError_t launch_i8_groups(const I8GroupsJob &j, hipStream_t s) {
#define CALL(T) groups_type<T>(j, s)
    I8_BY_TYPE(j.type, CALL)
#undef CALL
}

hipError_t launch_i8_back(const I8BackJob &j, hipStream_t s) {
#define CALL(T) back_type<T>(j, s)
    I8_BY_TYPE(j.type, CALL)
#undef CALL
}

}  // namespace sgemm
