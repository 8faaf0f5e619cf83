// Y = X W^T for a few rows X of floats and 4-bit weights W (N x K): the
// product of single tokens, bound by reading W once (0.53 bytes a weight).
//
// A workgroup takes up to 16 MT tokens, 8 KS slabs of K and a run of row
// tiles (mx4_thin.h).  Where K is longer than that, several workgroups share
// a row tile and write their sums to scratch memory, which a second kernel
// adds in K order: the same bits every time.  More than 64 tokens run 64 at a
// time.
//
// 1 x 4096 x 4096 bf16 takes 5.0 us (launch and latency), 13 x 5001 x 16384 fp32
// 17.0 and 4.1 for the joining: 4 us until the tokens are in registers, then 1.1
// for each of a workgroup's ten row tiles.
#include "mx4_thin.h"

namespace sgemm {
namespace {

constexpr int kMostTokens = 64;   // of one pass over the weights

// Whether the registers (128 a lane, without spills) let a CU hold two workgroups.
constexpr bool two_on_a_cu(int pieces, int ks, int mt) { return pieces == 1 ? mt == 1 || (mt == 2 && ks == 1) : ks * mt == 1; }
// Row tiles that a wave adds up at a time.
constexpr int group_of(int ks, int mt) { return mt > 1 ? 2 : ks == 4 ? 1 : 4; }

// Pieces by what they take of the registers while they are made: folded ones
// count as one, but an fp32 token is held whole first.
constexpr int register_pieces(int type, bool fold) { return fold && type != SGEMM_TYPE_F32 ? 1 : mx_pieces(type); }

struct Args {
    const void *x;
    int64_t ldx;
    MxWeights w;
    int M, N, K, per, parts;   // per: row tiles of a workgroup; parts: workgroups along K
    void *y;
    int64_t ldy;
    float *partial;                 // parts x M x pitch, if parts > 1
    int64_t pitch;
};

__device__ __forceinline__ int64_t weight_row(const Args &a, int tile, int m) {
    const int n = tile * 16 + m;
    return n < a.N ? n : a.N - 1;   // rows past N: computed, not stored
}

// Sums of token t, rows 16 tile + 4 quad + c where bit c of `rows` is set.
template <int TYPE>
__device__ __forceinline__ void store_sums(const Args &a, int part, int t, int tile, int quad, f32v4 v, int rows) {
    typedef typename MxType<TYPE>::T T;
    const int n = tile * 16 + 4 * quad;
    if (t >= a.M) return;
    if (a.parts > 1) {
        mx_store_rows(a.partial + ((int64_t)part * a.M + t) * a.pitch + n, v, rows);
        return;
    }
    T *y = (T *)a.y + t * a.ldy + n;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (n + c < a.N && (rows >> c & 1)) y[c] = MxType<TYPE>::from(v[c]);
}

template <int TYPE, int KS, int MT, int G, bool FOLD>
__global__ __launch_bounds__(kThinThreads, two_on_a_cu(register_pieces(TYPE, FOLD), KS, MT) ? 4 : 2) void linear_kernel(Args a) {
    typedef typename MxType<TYPE>::T T;
    typedef MxTokens<TYPE, mx_pieces(TYPE), KS, kThinWaves, MT, FOLD> Tokens;
    typedef MxStream<1, G, KS, kThinWaves, false> Stream;
    __shared__ __attribute__((aligned(16))) f32v4 red[kThinSums<G, MT>];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int part = blockIdx.x % a.parts, first = blockIdx.x / a.parts * a.per, m0 = blockIdx.y * 16 * MT;
    const int tiles = (a.N + 15) / 16, end = first + a.per < tiles ? first + a.per : tiles;
    const int slab0 = (part * kThinWaves + wave) * KS;
    const auto row_of = [&](int tile, int m) { return weight_row(a, tile, m); };
    Tokens x;
    const T *row[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int t = m0 + mt * 16 + x.token();
        row[mt] = x.token() >= 0 && t < a.M ? (const T *)a.x + t * a.ldx : nullptr;
    }
    x.load(row, slab0, a.K, lane >> 4);
    Stream stream;
    stream.begin(a.w, slab0, first, end, row_of);
    bool odd = false;
    stream.run(x, a.w, slab0, first, end, red, nullptr, true, true, odd, row_of, [&](int tile, int mt, int l, const f32v4(&v)[1], int rows) {
        store_sums<TYPE>(a, part, m0 + mt * 16 + (l & 15), tile, l >> 4, v[0], rows);
    });
    if (__builtin_expect(odd, 0)) {   // weights beyond the largest float?
        const Args b = mx_arguments<Args>();
        const int part = blockIdx.x % b.parts, first = blockIdx.x / b.parts * b.per, m0 = blockIdx.y * 16 * MT;
        const int tiles = (b.N + 15) / 16, end = first + b.per < tiles ? first + b.per : tiles;
        Stream::template mend<MT, Tokens::kTokens>(
            b.w, part * kThinWaves * KS, (part + 1) * kThinWaves * KS, first, end, [&](int tile, int m) { return weight_row(b, tile, m); },
            [&](int mt, int t16, int column) {
                const int t = m0 + mt * 16 + t16;
                return t < b.M && column < b.K ? MxType<TYPE>::load((const T *)b.x + t * b.ldx + column) : 0.0f;
            },
            [&](int tile, int mt, int l, const f32v4(&v)[1], int rows) {
                store_sums<TYPE>(b, part, m0 + mt * 16 + (l & 15), tile, l >> 4, v[0], rows);
            });
    }
}

// Adds the parts; a thread takes one value.
template <int TYPE>
__global__ __launch_bounds__(256) void join_kernel(Args a) {
    const int n = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (n >= a.N) return;
    const float *p = a.partial + t * a.pitch + n;
    float sum = *p;
    for (int k = 1; k < a.parts; ++k) sum += p[k * a.M * a.pitch];
    ((typename MxType<TYPE>::T *)a.y)[t * a.ldy + n] = MxType<TYPE>::from(sum);
}

// How a pass of up to 64 tokens runs.
struct Shape {
    int mt, ks, parts;   // token tiles of a workgroup, slabs of a wave, workgroups along K
    bool fold;
};
Shape shape_of(int M, int K, int type) {
    Shape s;
    s.fold = type == SGEMM_TYPE_F16 ? M <= 8 : type == SGEMM_TYPE_F32 && M <= 5;
    s.mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    if (type == SGEMM_TYPE_F32 && s.mt > 2) s.mt = 2;   // (four tiles would take 192 registers)
    // As many slabs as hold K, up to what the registers hold.
    const int most = type == SGEMM_TYPE_F32                ? (s.mt == 1 ? 2 : 1)
                     : type == SGEMM_TYPE_BF16 || s.fold ? (s.mt == 1 ? 4 : 2)
                                                         : (s.mt < 4 ? 2 : 1);
    const int need = (mx_slabs(K) + kThinWaves - 1) / kThinWaves;
    s.ks = need >= most ? most : need > 2 ? 4 : need > 1 ? 2 : 1;
    s.parts = (mx_slabs(K) + kThinWaves * s.ks - 1) / (kThinWaves * s.ks);
    if (s.parts < 1) s.parts = 1;
    return s;
}

template <int TYPE, int KS, int MT, bool FOLD>
hipError_t launch_shape(Args a, hipStream_t s) {
    constexpr int G = group_of(KS, MT);
    // Workgroups: as many as the CUs hold at once.
    constexpr int kWant = two_on_a_cu(register_pieces(TYPE, FOLD), KS, MT) ? 512 : 256;
    const int tiles = (a.N + 15) / 16, groups = kWant / a.parts > 0 ? kWant / a.parts : 1;
    a.per = mx_share(tiles, groups < tiles ? groups : tiles, 1);
    const int row_groups = (tiles + a.per - 1) / a.per;
    void *params[] = {&a};
    hipError_t e = hipLaunchKernel((const void *)linear_kernel<TYPE, KS, MT, G, FOLD>,
                                   dim3((unsigned)(row_groups * a.parts), (unsigned)((a.M + 16 * MT - 1) / (16 * MT))),
                                   dim3(kThinThreads), params, 0, s);
    if (e != hipSuccess || a.parts == 1) return e;
    return hipLaunchKernel((const void *)join_kernel<TYPE>, dim3((unsigned)((a.N + 255) / 256), (unsigned)a.M), dim3(256), params,
                           0, s);
}

template <int TYPE, int MT, bool FOLD>
hipError_t launch_tokens(const Args &a, int ks, hipStream_t s) {
    constexpr int P = register_pieces(TYPE, FOLD);
    if constexpr (P == 1 && MT == 1)
        if (ks == 4) return launch_shape<TYPE, 4, MT, FOLD>(a, s);
    if constexpr (P == 1 || (P == 2 && MT < 4) || (P == 3 && MT == 1))
        if (ks == 2) return launch_shape<TYPE, 2, MT, FOLD>(a, s);
    return launch_shape<TYPE, 1, MT, FOLD>(a, s);
}

template <int TYPE>
hipError_t launch_type(const MxLinearJob &j, hipStream_t s) {
    const int64_t esize = TYPE == SGEMM_TYPE_F32 ? 4 : 2;
    for (int64_t m = 0; m < j.M; m += kMostTokens) {
        Args a;
        a.M = j.M - m < kMostTokens ? (int)(j.M - m) : kMostTokens;
        a.x = (const char *)j.x + m * j.ldx * esize;
        a.ldx = j.ldx;
        a.w = mx_weights(j.codes, j.scales, j.N, j.K);
        a.N = j.N;
        a.K = j.K;
        a.y = (char *)j.y + m * j.ldy * esize;
        a.ldy = j.ldy;
        const Shape shape = shape_of(a.M, a.K, TYPE);
        a.parts = shape.parts;
        a.partial = j.scratch;
        a.pitch = ((int64_t)j.N + 15) / 16 * 16;
        hipError_t e = hipErrorInvalidValue;
        if (shape.fold) {
            if constexpr (TYPE != SGEMM_TYPE_BF16) e = launch_tokens<TYPE, 1, true>(a, shape.ks, s);
        } else if (shape.mt == 1) {
            e = launch_tokens<TYPE, 1, false>(a, shape.ks, s);
        } else if (shape.mt == 2) {
            e = launch_tokens<TYPE, 2, false>(a, shape.ks, s);
        } else {
            if constexpr (TYPE != SGEMM_TYPE_F32) e = launch_tokens<TYPE, 4, false>(a, shape.ks, s);
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t mx4_linear_scratch(int M, int N, int K, int type) {
    // The passes: full ones of 64 tokens, and the last.
    int64_t most = 0;
    const int sizes[] = {M < kMostTokens ? M : kMostTokens, M % kMostTokens};
    for (int m : sizes) {
        if (m == 0) continue;
        const int64_t parts = shape_of(m, K, type).parts;
        const int64_t bytes = parts > 1 ? parts * m * (((int64_t)N + 15) / 16 * 16) * 4 : 0;
        most = bytes > most ? bytes : most;
    }
    return most;
}

hipError_t launch_mx4_linear(const MxLinearJob &j, hipStream_t s) {
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_type<SGEMM_TYPE_F32>(j, s);
    case SGEMM_TYPE_F16: return launch_type<SGEMM_TYPE_F16>(j, s);
    case SGEMM_TYPE_BF16: return launch_type<SGEMM_TYPE_BF16>(j, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace sgemm
