// The product of a few rows of 8-bit integers ("tokens") with many ("weights"),
// and the same of float tokens that are quantised on the way.
//
// Bound by reading the weights once.  A wave takes 8 G rows of weights and every
// wk-th block of 128 along K; the waves that share rows add their sums, exact
// integers, in LDS at the end.  One load is 8 rows x 128 bytes: whole lines of
// memory.  On v_mfma_i32_16x16x64_i8, whose first operand has 16 rows of 64
// bytes, row 2 r + p takes half p of the block of row r, and column 8 c + t of
// the second takes half c of token t: entries with p = c are parts of the result
// (of row r and token t), the others are dropped.  Half of the matrix work is
// wasted, which is idle otherwise.
//
// In a graph, different weights in turn, one token: 4096 x 4096 5.9 us (16.8 MB: 3.3
// at 5.1 TB/s), from bf16 7.4; 16384 x 4096 14.4 (67 MB: 13.1); 5001 x 16384 21.4 (82
// MB: 16.0).  Eight: 6.5, 9.5, 15.4, 23.4.
#include "i8.h"

namespace sgemm {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
template <int TYPE>
constexpr int kKept = TYPE == SGEMM_TYPE_F32 ? 2 : 4;   // eights of a token that a lane keeps while it looks for the largest

struct Args {
    const int8_t *w;
    const float *sw;
    const int8_t *x;       // tokens as 8-bit integers, with scales sx; or
    const float *sx;
    const void *xf;        // as floats
    int64_t ldx;
    int rows, tokens, blocks;   // blocks of 128 along K
    int k;
    int wk;                // waves that share rows: a power of two
    int wt;                // waves that quantise a token: a power of two
    float alpha, beta;
    int type;
    void *c;
    int64_t by_row, by_token;   // elements from one row of weights (token) to the next in the result
};

template <int TYPE>
__device__ __forceinline__ void put(const Args &g, int64_t at, float v) {
    auto *p = (typename MxType<TYPE>::T *)g.c + at;
    if (g.beta != 0.0f) v += g.beta * MxType<TYPE>::load(p);
    *p = MxType<TYPE>::from(v);
}

// Quantises the float tokens into LDS, rows of `ld` bytes, and their scales.
// All tokens at once: wt waves, a power of two, take one.
template <int TYPE>
__device__ __forceinline__ void quantise(const Args &g, int8_t *q, int ld, float *scale, uint32_t *most) {
    typedef typename MxType<TYPE>::T E;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wt = g.wt, t = wave / wt, c0 = 8 * ((wave & (wt - 1)) * 64 + lane), step = 512 * wt;
    const bool real = t < g.tokens;
    const E *x = (const E *)g.xf + (real ? t : 0) * g.ldx;
    const int kp = g.blocks * 128;
    // A token of up to kKept eights a lane stays in registers between the passes.
    constexpr int KEPT = kKept<TYPE>;
    I8Raw<TYPE> raw[KEPT];
    const auto load = [&](int c, uint32_t m) {
        i8_load_row<TYPE>(x, c, step, real ? g.k : 0, raw);
#pragma unroll
        for (int i = 0; i < KEPT; ++i) {
            float v[8];
            raw[i].get(v);
            m = i8_max(m, i8_max8(v));
        }
        return m;
    };
    const int whole = step * KEPT;
    uint32_t m = 0;
    for (int c = c0 + whole; c < g.k; c += whole) m = load(c, m);
    m = load(c0, m);
    m = i8_max16(m);
    m = i8_max(m, __shfl_xor(m, 16, 64));
    m = i8_max(m, __shfl_xor(m, 32, 64));
    if (lane == 0) most[wave] = m;
    __syncthreads();
    if (real) {
        for (int i = t * wt; i < (t + 1) * wt; ++i) m = i8_max(m, most[i]);
        const float s = i8_scale(m, kI8Levels), inv = 1.0f / s;
        for (int c = c0; c < kp; c += whole) {
            if (c > c0) load(c, 0);
#pragma unroll
            for (int i = 0; i < KEPT; ++i)
                if (c + i * step < kp) {
                    float v[8];
                    raw[i].get(v);
                    *(uint2 *)(q + t * ld + c + i * step) = i8_nearest8(v, s, inv);
                }
        }
        if (lane == 0) scale[t] = s;
    }
    __syncthreads();
}

// FLOATS: the type of float tokens, or -1.
template <int G, int FLOATS>
__global__ __launch_bounds__(kThreads, 4) void i8_thin_kernel(Args g) {
    extern __shared__ __attribute__((aligned(16))) int8_t lds[];
    __shared__ float scale[kI8ThinRows];
    __shared__ uint32_t most[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = wave & (g.wk - 1), set = wave / g.wk, sets = kWaves / g.wk;
    const int row0 = (blockIdx.x * sets + set) * 8 * G;
    const int64_t kp = (int64_t)g.blocks * 128;
    const int8_t *w[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int r = row0 + 8 * i + ((lane & 15) >> 1);
        w[i] = g.w + (r < g.rows ? r : g.rows - 1) * kp + 16 * (4 * (lane & 1) + (lane >> 4));
    }
    const int quad = 16 * (4 * ((lane >> 3) & 1) + (lane >> 4));
    const int xld = (int)kp + 16;    // of a token in LDS
    struct Block {
        i32v4 w[G], x;
    };
    const int token = (lane & 7) < g.tokens ? lane & 7 : g.tokens - 1;
    const int8_t *x = FLOATS >= 0 ? lds + token * xld + quad : g.x + token * kp + quad;
    i32v4 acc[G];
#pragma unroll
    for (int i = 0; i < G; ++i) acc[i] = i32v4{0, 0, 0, 0};
    const auto load = [&](Block &b, int at) {
#pragma unroll
        for (int i = 0; i < G; ++i) b.w[i] = *(const i32v4 *)(w[i] + (int64_t)at * 128);
        if constexpr (FLOATS < 0) b.x = *(const i32v4 *)(x + (int64_t)at * 128);
    };
    const auto multiply = [&](Block &b, int at) {
        if constexpr (FLOATS >= 0) b.x = *(const i32v4 *)(x + at * 128);
#pragma unroll
        for (int i = 0; i < G; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b.w[i], b.x, acc[i], 0, 0, 0);
    };
    constexpr int U = 4;   // blocks in flight
    Block b[U];
    const int step = g.wk;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (kw + u * step < g.blocks) load(b[u], kw + u * step);
    if constexpr (FLOATS >= 0) quantise<FLOATS>(g, lds, xld, scale, most);
    for (int at = kw; at < g.blocks; at += U * step) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int here = at + u * step, next = here + U * step;
            if (here < g.blocks) multiply(b[u], here);
            if (next < g.blocks) load(b[u], next);
        }
    }
    // Sums of the waves that share rows, and of the two halves of a block.  (A
    // lane reads one row's, and those of neighbouring rows lie 16 or 64 words apart:
    // with one token and 4096 columns 48 of a workgroup's 112 conflict cycles.  LDS
    // is busy in 4% of the kernel's cycles, conflicts in 19% of those.)
    __syncthreads();
    int *red = (int *)lds;    // [set][kw][G][row parity][lane]
    {
        const int c = (lane >> 3) & 1;
        int *mine = red + wave * (G * 128) + lane;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            mine[i * 128] = c ? acc[i][1] : acc[i][0];
            mine[i * 128 + 64] = c ? acc[i][3] : acc[i][2];
        }
    }
    __syncthreads();
    const int per = sets * 8 * G, all = per * g.tokens, first = blockIdx.x * per;
    for (int o = tid; o < all; o += kThreads) {
        // Next to each other in the result: rows, or tokens.
        const bool across = g.by_row == 1;
        const int r = across ? o % per : o / g.tokens, t = across ? o / per : o - r * g.tokens;
        const int row = first + r;
        if (row >= g.rows) continue;
        const int s = r / (8 * G), i = (r >> 3) % G, r8 = r & 7;
        const int *p = red + s * g.wk * (G * 128) + i * 128 + 64 * (r8 & 1) + 16 * (r8 >> 1) + t;
        int sum = 0;
        for (int k = 0; k < g.wk; ++k) sum += p[k * (G * 128)] + p[k * (G * 128) + 8];
        const float sx = FLOATS >= 0 ? scale[t] : g.sx ? g.sx[t] : 1.0f, sw = g.sw ? g.sw[row] : 1.0f;
        const float v = g.alpha * i8_scaled((float)sum, sx, sw);
        const int64_t to = row * g.by_row + t * g.by_token;
        if (g.type == SGEMM_TYPE_F32) put<SGEMM_TYPE_F32>(g, to, v);
        else if (g.type == SGEMM_TYPE_BF16) put<SGEMM_TYPE_BF16>(g, to, v);
        else put<SGEMM_TYPE_F16>(g, to, v);
    }
}

template <int G, int FLOATS>
hipError_t launch(Args g, hipStream_t s) {
    g.wk = 1;
    while (g.wk < kWaves && 2 * g.wk <= g.blocks) g.wk *= 2;
    g.wt = kWaves;
    while (g.wt > 1 && kWaves / g.wt < g.tokens) g.wt /= 2;
    const int per = kWaves / g.wk * 8 * G;
    const int red = kWaves * G * 512, tokens = FLOATS >= 0 ? g.tokens * (g.blocks * 128 + 16) : 0;
    void *params[] = {&g};
    return hipLaunchKernel((const void *)i8_thin_kernel<G, FLOATS>, dim3((unsigned)((g.rows + per - 1) / per)), dim3(kThreads), params,
                           red > tokens ? red : tokens, s);
}

template <int FLOATS>
hipError_t launch_rows(const Args &g, int num_cus, hipStream_t s) {
    // Enough workgroups for every CU; else more rows for each token that is read.
    return (int64_t)g.rows <= 16 * 2 * num_cus ? launch<2, FLOATS>(g, s) : launch<4, FLOATS>(g, s);
}

}  // namespace

// Tiles of 32 x 32 stream the largest weights faster (16384 x 16384, one token:
// 51.6 us against 57.3; 28672 x 8192 44.4 against 49.4; 12000 x 8192, 98 MB, the
// same; 8192 x 4096: 9.5 against 8.7).
bool i8_thin_takes(int M, int N, int K) {
    const int few = M < N ? M : N, many = M < N ? N : M;
    return few <= kI8ThinRows && many * i8_ld(K) <= 1LL << 27;
}

// Every workgroup quantises the float tokens anew: with few values that costs
// less than a kernel of its own (4096 x 4096, one token: 7.4 us against 8.8, four:
// 7.9 against 9.0, eight the same; 5001 x 16384, one: 22.2 against 25.2, four: 28.8
// against 26.2).
bool i8_thin_takes_floats(int M, int N, int K) {
    return M <= kI8ThinRows && M * i8_ld(K) <= 16384 && N * i8_ld(K) <= 1LL << 27;
}

hipError_t launch_i8_thin(const I8GemmJob &j, const void *floats, int64_t ldx, int num_cus, hipStream_t s) {
    Args g{};
    const bool turned = !floats && j.N < j.M;   // the fewer rows are the tokens
    g.w = turned ? j.a : j.b, g.sw = turned ? j.sa : j.sb, g.x = turned ? j.b : j.a, g.sx = turned ? j.sb : j.sa;
    g.xf = floats, g.ldx = ldx;
    g.rows = turned ? j.M : j.N, g.tokens = turned ? j.N : j.M;
    g.k = j.K, g.blocks = (int)(i8_ld(j.K) / 128);
    g.alpha = j.alpha, g.beta = j.beta, g.type = j.type, g.c = j.c;
    g.by_row = turned ? j.ldc : 1, g.by_token = turned ? 1 : j.ldc;
    if (floats) {
        switch (j.type) {
        case SGEMM_TYPE_F32: return launch_rows<SGEMM_TYPE_F32>(g, num_cus, s);
        case SGEMM_TYPE_BF16: return launch_rows<SGEMM_TYPE_BF16>(g, num_cus, s);
        case SGEMM_TYPE_F16: return launch_rows<SGEMM_TYPE_F16>(g, num_cus, s);
        default: return hipErrorInvalidValue;
        }
    }
    return launch_rows<-1>(g, num_cus, s);
}

}  // namespace sgemm
