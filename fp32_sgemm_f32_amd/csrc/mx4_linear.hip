// Y = X W^T for a few rows X of floats and 4-bit weights W (N x K): the
// product of single tokens, bound by reading W once (0.53 bytes a weight).
//
// A workgroup takes up to 16 MT tokens, 8 KS slabs of K and a run of row
// tiles (mx4_thin.h).  Where K is longer than that, several workgroups share
// a row tile and write their sums to scratch memory, which a second kernel
// adds in K order: the same bits every time.  More than 64 tokens run 64 at a
// time.
#include "mx4_thin.h"

namespace sgemm {
namespace {

constexpr int kMostTokens = 64;   // of one pass over the weights

// Whether the registers (128 a lane, without spills) let a CU hold two workgroups.
constexpr bool two_on_a_cu(int pieces, int ks, int mt) { return pieces == 1 ? mt == 1 || (mt == 2 && ks == 1) : ks * mt == 1; }
// Row tiles that a wave adds up at a time.
constexpr int group_of(int ks, int mt) { return mt > 1 ? 2 : ks == 4 ? 1 : 4; }

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

template <int TYPE, int KS, int MT, int G>
__global__ __launch_bounds__(kThinThreads, two_on_a_cu(mx_pieces(TYPE), KS, MT) ? 4 : 2) void linear_kernel(Args a) {
    typedef typename MxType<TYPE>::T T;
    __shared__ __attribute__((aligned(16))) f32v4 red[kThinSums<G, MT>];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int part = blockIdx.x % a.parts, first = blockIdx.x / a.parts * a.per, m0 = blockIdx.y * 16 * MT;
    const int tiles = (a.N + 15) / 16, end = first + a.per < tiles ? first + a.per : tiles;
    const int slab0 = (part * kThinWaves + wave) * KS;
    const auto row_of = [&](int tile, int m) -> int64_t {
        const int n = tile * 16 + m;
        return n < a.N ? n : a.N - 1;   // rows past N: computed, not stored
    };
    const T *row[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int t = m0 + mt * 16 + (lane & 15);
        row[mt] = t < a.M ? (const T *)a.x + t * a.ldx : nullptr;
    }
    MxTokens<TYPE, mx_pieces(TYPE), KS, kThinWaves, MT> x;
    x.load(row, slab0, a.K, lane >> 4);
    MxStream<1, G, KS, kThinWaves, false> stream;
    stream.begin(a.w, slab0, first, end, row_of);
    stream.run(
        x, a.w, slab0, first, end, red, nullptr, true, true, row_of,
        [&](int tile, int mt, int l, const f32v4(&v)[1]) {
            const int t = m0 + mt * 16 + (l & 15), n = tile * 16 + 4 * (l >> 4);
            if (t >= a.M) return;
            if (a.parts > 1) {
                *(f32v4 *)(a.partial + ((int64_t)part * a.M + t) * a.pitch + n) = v[0];
                return;
            }
            T *y = (T *)a.y + t * a.ldy + n;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (n + c < a.N) y[c] = MxType<TYPE>::from(v[0][c]);
        });
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

// Slabs that a wave keeps: as many as hold K, up to `most` (the registers).
int kept_slabs(int K, int most) {
    const int need = (mx_slabs(K) + kThinWaves - 1) / kThinWaves;
    return need >= most ? most : need > 2 ? 4 : need > 1 ? 2 : 1;
}
// That most, for 16 mt tokens.
int most_slabs(int type, int mt) {
    if (type == SGEMM_TYPE_BF16) return mt == 1 ? 4 : 2;
    if (type == SGEMM_TYPE_F16) return mt < 4 ? 2 : 1;
    return mt == 1 ? 2 : 1;
}
// Token tiles of a workgroup; fp32 stops at 2 (four would take 192 registers).
int token_tiles(int M, int type) {
    const int mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    return type == SGEMM_TYPE_F32 && mt > 2 ? 2 : mt;
}
int k_parts(int M, int K, int type) {
    const int ks = kept_slabs(K, most_slabs(type, token_tiles(M, type)));
    const int parts = (mx_slabs(K) + kThinWaves * ks - 1) / (kThinWaves * ks);
    return parts > 0 ? parts : 1;
}

template <int TYPE, int KS, int MT>
hipError_t launch_shape(Args a, hipStream_t s) {
    constexpr int G = group_of(KS, MT);
    // Workgroups: as many as the CUs hold at once.
    constexpr int kWant = two_on_a_cu(mx_pieces(TYPE), KS, MT) ? 512 : 256;
    const int tiles = (a.N + 15) / 16, groups = kWant / a.parts > 0 ? kWant / a.parts : 1;
    a.per = mx_share(tiles, groups < tiles ? groups : tiles, 1);
    const int row_groups = (tiles + a.per - 1) / a.per;
    void *params[] = {&a};
    hipError_t e = hipLaunchKernel((const void *)linear_kernel<TYPE, KS, MT, G>,
                                   dim3((unsigned)(row_groups * a.parts), (unsigned)((a.M + 16 * MT - 1) / (16 * MT))),
                                   dim3(kThinThreads), params, 0, s);
    if (e != hipSuccess || a.parts == 1) return e;
    return hipLaunchKernel((const void *)join_kernel<TYPE>, dim3((unsigned)((a.N + 255) / 256), (unsigned)a.M), dim3(256), params,
                           0, s);
}

template <int TYPE, int MT>
hipError_t launch_tokens(const Args &a, hipStream_t s) {
    const int ks = kept_slabs(a.K, most_slabs(TYPE, MT));
    if constexpr (TYPE == SGEMM_TYPE_BF16 && MT == 1)
        if (ks == 4) return launch_shape<TYPE, 4, MT>(a, s);
    if constexpr (!(TYPE == SGEMM_TYPE_F16 && MT == 4) && !(TYPE == SGEMM_TYPE_F32 && MT > 1))
        if (ks == 2) return launch_shape<TYPE, 2, MT>(a, s);
    return launch_shape<TYPE, 1, MT>(a, s);
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
        a.parts = k_parts(a.M, a.K, TYPE);
        a.partial = j.scratch;
        a.pitch = ((int64_t)j.N + 15) / 16 * 16;
        const int mt = token_tiles(a.M, TYPE);
        hipError_t e;
        if (mt == 1) e = launch_tokens<TYPE, 1>(a, s);
        else if (mt == 2) e = launch_tokens<TYPE, 2>(a, s);
        else if constexpr (TYPE != SGEMM_TYPE_F32) e = launch_tokens<TYPE, 4>(a, s);
        else e = hipErrorInvalidValue;
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
        const int64_t parts = k_parts(m, K, type);
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
