// A mixture-of-experts layer for a few tokens, experts in 4 bits:
//
//   l = x R^T                         router logits of a token (E experts)
//   S = the `top` largest of l        lower index first on equal logits
//   p_e = exp(l_e - max) / sum        sum over S (norm) or over all experts
//   y = sum over e in S of p_e D_e (silu(G_e x) * (U_e x))
//
// G_e and U_e are rows [2 e F, 2 e F + F) and [2 e F + F, 2 e F + 2 F) of
// `up` (2 E F x H), D_e rows [e H, e H + H) of `down` (E H x F).
//
// Bound by reading the chosen experts once: 3 F H 0.53 bytes each.  48 tokens, 8
// of 128 experts of 4096 x 1536, bf16: 266 us; `up` reads 816 MB in 146 (5.6
// TB/s), `down` 408 MB in 113 (3.6).  One token, 8 of 64 experts of 2048 x 768:
// 17.5 us in a graph, latencies one after another.
//
// Logits are summed in 64 bits: which expert is chosen must not hang on the
// order of a sum.  The inner activations enter the second product as three
// bf16 pieces, 24 bits, whatever the type of the tokens: nothing is rounded
// between a token and its result but fp32 sums.  Every sum has a fixed order:
// results repeat bit for bit.
//
// Few choices (tokens * top <= kFew): three kernels.
//   logits    a wave takes an expert
//   up (FEW)  a workgroup takes one choice and a run of inner columns; it
//             ranks the token's experts by itself (a kernel for that alone
//             costs more than all of them doing it)
//   down_few  a workgroup takes 16 rows of the output and all choices: its
//             waves share the (choice, slab) list evenly and add p_e times
//             their part into sums of their own, added in wave order
// (2 tokens, 8 of 64 experts of 2048 x 768: 25.1 us so, 29.1 by the five below;
// 4 tokens, before folding, 45 against 36.)
// More: five.
//   logits, choose
//   up        a workgroup takes an expert and a run of inner columns, for all
//             tokens of the expert, 16 at a time (mx4_thin.h)
//   down      the same for rows of the output; writes each choice's part
//   join      adds a token's parts, times their weights, best first
#include <type_traits>

#include "mx4_thin.h"

namespace sgemm {
namespace {

constexpr int kFew = 16;
// Whether the registers (128 a lane, without spills) let a CU hold two
// workgroups, which hide each other's beginnings and meetings, and the row
// tiles that a wave adds up at a time: as many loads in flight as the registers
// hold.  (Two pieces of two slabs spilled at two workgroups: `up` of fp16, the
// layer for 48 tokens, 8 of 128 experts, 4096 x 1536: 365 us so, 336 with one.)
constexpr bool two_on_a_cu(int pieces, int ks, bool few) { return ks <= 2 && pieces * ks <= (few ? 2 : 3); }
// Pieces by what they take of the registers while they are made: folded ones
// count as one, but an fp32 token is held whole first.
constexpr int register_pieces(int type, bool fold) { return fold && type != SGEMM_TYPE_F32 ? 1 : mx_pieces(type); }
constexpr int group_of(int pieces, int ks, bool few) {
    return few ? 2 : two_on_a_cu(pieces, ks, few) ? (ks == 1 && pieces <= 2 ? 4 : 2) : pieces == 1 ? 4 : 2;
}
constexpr int kActPieces = 3;   // of an inner activation

// Scratch memory, every part 256-byte aligned.
struct Scratch {
    double *logits;   // tokens x experts
    int *chosen;      // tokens x top
    float *weight;    // tokens x top
    uint16_t *act;    // kActPieces x (tokens * top) x ld_act (inner rounded up to 16), zeros beyond inner
    float *part;      // (tokens * top) x ld_part; not with few choices
    int64_t ld_act, ld_part, bytes;
};

Scratch layout(char *p, int tokens, int hidden, int inner, int experts, int top) {
    Scratch s;
    int64_t at = 0;
    const auto take = [&](int64_t n) { const int64_t here = at; at += (n + 255) & ~(int64_t)255; return p + here; };
    const int64_t all = (int64_t)tokens * top;
    s.ld_act = ((int64_t)inner + 15) / 16 * 16;
    s.ld_part = ((int64_t)hidden + 15) / 16 * 16;
    s.logits = (double *)take((int64_t)tokens * experts * 8);
    s.chosen = (int *)take(all * 4);
    s.weight = (float *)take(all * 4);
    s.act = (uint16_t *)take(kActPieces * all * s.ld_act * 2);
    s.part = (float *)take(all > kFew ? all * s.ld_part * 4 : 0);
    s.bytes = at;
    return s;
}

// ---- router ----

// A wave takes one expert and TT tokens.
template <int TYPE, int TT>
__global__ __launch_bounds__(256) void logits_kernel(MxMoeJob j, Scratch s) {
    typedef typename MxType<TYPE>::T T;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 4 + wave, t0 = blockIdx.y * TT;
    const T *r = (const T *)j.router + (e < j.experts ? e : 0) * j.ldr;
    const T *x[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t] = (const T *)j.x + (t0 + t < j.tokens ? t0 + t : t0) * j.ldx;
    double sum[TT] = {};
    auto add = [&](const float (&w)[8], const float (&v)[TT][8]) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[t] = fma((double)w[i], (double)v[t][i], sum[t]);
    };
    int h = 8 * lane;
    // Two steps' loads in flight.
    for (; h + 512 + 8 <= j.hidden; h += 1024) {
        float w[2][8], v[2][TT][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            mx_load8<TYPE>(r + h + 512 * k, w[k]);
#pragma unroll
            for (int t = 0; t < TT; ++t) mx_load8<TYPE>(x[t] + h + 512 * k, v[k][t]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) add(w[k], v[k]);
    }
    for (; h < j.hidden; h += 512) {
        float w[8], v[TT][8];
        mx_load_edge8<TYPE>(r, h, j.hidden, w);
#pragma unroll
        for (int t = 0; t < TT; ++t) mx_load_edge8<TYPE>(x[t], h, j.hidden, v[t]);
        add(w, v);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum[t] += __shfl_xor(sum[t], off, 64);
        if (lane == 0 && e < j.experts && t0 + t < j.tokens) s.logits[(int64_t)(t0 + t) * j.experts + e] = sum[t];
    }
}

// A logit as an integer of the same order: NaN above all, -0 equal to 0.
__device__ __forceinline__ int64_t order_key(double v) {
    if (v != v) return INT64_MAX;
    const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
    return b < 0 ? b ^ INT64_MAX : b;
}

struct Choice {
    int64_t key[SGEMM_MX4_MAX_EXPERTS];
    int rank[SGEMM_MX4_MAX_EXPERTS];
    float part[kThinWaves];
    float value[SGEMM_MX4_MAX_TOP];    // exponentials
    int expert[SGEMM_MX4_MAX_TOP];
};

// Ranks a token's experts, by the whole workgroup: an expert's rank is the
// number of experts before it, counted in as many pieces as there are threads
// for.
__device__ __forceinline__ void rank_experts(const MxMoeJob &j, const double *l, Choice &c) {
    const int tid = threadIdx.x, n = j.experts;
    for (int e = tid; e < n; e += kThinThreads) c.key[e] = order_key(l[e]), c.rank[e] = 0;
    __syncthreads();
    const int pieces = n < kThinThreads ? kThinThreads / n : 1;
    for (int i = tid; i < n * pieces; i += kThinThreads) {
        const int e = i % n, piece = i / n, from = n * piece / pieces, to = n * (piece + 1) / pieces;
        const int64_t mine = c.key[e];
        int before = 0;
#pragma unroll 8
        for (int o = from; o < to; ++o) before += c.key[o] > mine || (c.key[o] == mine && o < e);
        if (before > 0) atomicAdd(&c.rank[e], before);   // whole numbers: any order
    }
    __syncthreads();
    for (int e = tid; e < n; e += kThinThreads) {
        const int r = c.rank[e];
        if (r < j.top) c.expert[r] = e;
    }
    __syncthreads();
}

// Writes the choices of token t, best first, and their weights, after
// rank_experts.
__device__ __forceinline__ void write_choice(const MxMoeJob &j, const Scratch &s, int t, const double *l, Choice &c) {
    const int tid = threadIdx.x, n = j.experts;
    const double best = l[c.expert[0]];
    float total = 0.0f;
    for (int e = tid; e < n; e += kThinThreads) {
        const float v = expf((float)(l[e] - best));
        total += v;
        if (c.rank[e] < j.top) c.value[c.rank[e]] = v;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) total += __shfl_xor(total, off, 64);
    if ((tid & 63) == 0) c.part[tid >> 6] = total;
    __syncthreads();
    if (tid < j.top) {
        float sum = 0.0f;
        if (j.norm)
            for (int i = 0; i < j.top; ++i) sum += c.value[i];
        else
            for (int i = 0; i < kThinWaves; ++i) sum += c.part[i];
        s.chosen[t * j.top + tid] = c.expert[tid];
        s.weight[t * j.top + tid] = c.value[tid] / sum;
    }
}

__global__ __launch_bounds__(kThinThreads) void choose_kernel(MxMoeJob j, Scratch s) {
    __shared__ Choice c;
    const double *l = s.logits + (int64_t)blockIdx.x * j.experts;
    rank_experts(j, l, c);
    write_choice(j, s, blockIdx.x, l, c);
}

// The expert of a workgroup and its choices, in any order (a token's result
// does not depend on its place).  blockIdx.y is the expert, or, with fewer
// choices than experts, a choice, which stands for its expert if none before
// it does (4 tokens, 8 of 64 experts of 2048 x 768: 35.1 us, 35.9 with a row of
// workgroups for every expert).
struct Listed {
    int list[SGEMM_MX4_MAX_TOKENS], token[SGEMM_MX4_MAX_TOKENS], count, earlier, expert;
};
__device__ __forceinline__ int list_tokens(const MxMoeJob &j, const int *chosen, int &e, Listed &l) {
    const int all = j.tokens * j.top;
    const bool by_choice = all < j.experts;
    e = by_choice ? chosen[blockIdx.y] : (int)blockIdx.y;
    if (threadIdx.x == 0) l.count = 0, l.earlier = 0, l.expert = e;
    __syncthreads();
    for (int a = threadIdx.x; a < all; a += kThinThreads)
        if (chosen[a] == e) {
            const int i = atomicAdd(&l.count, 1);
            l.list[i] = a, l.token[i] = a / j.top;
            if (by_choice && a < (int)blockIdx.y) l.earlier = 1;
        }
    __syncthreads();
    return l.earlier ? 0 : l.count;
}
int expert_rows(const MxMoeJob &j) { return j.tokens * j.top < j.experts ? j.tokens * j.top : j.experts; }

// Arguments of the kernels that stream weights.
struct StreamArgs {
    MxMoeJob j;
    Scratch s;
    MxWeights w;
    int per;   // row tiles of a workgroup
};

// ---- up ----

// Row tiles come in pairs: 16 rows of the gate, the same 16 of U.
inline __host__ __device__ int up_tiles(const MxMoeJob &j) { return 2 * ((j.inner + 15) / 16); }
__device__ __forceinline__ int64_t up_row(const MxMoeJob &j, int e, int tile, int m) {
    const int f = (tile >> 1) * 16 + m;
    return (int64_t)2 * e * j.inner + (f < j.inner ? f : j.inner - 1) + (tile & 1 ? j.inner : 0);
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// Inner activations f .. f + 3 of choice a, those whose bits are set in `rows`.
__device__ __forceinline__ void store_activations(const MxMoeJob &j, const Scratch &s, int a, int f, f32v4 g, f32v4 u, int rows) {
    uint16_t p[4][kActPieces];
#pragma unroll
    for (int c = 0; c < 4; ++c) mx_split<kActPieces>(f + c < j.inner ? silu(g[c]) * u[c] : 0.0f, p[c]);
#pragma unroll
    for (int k = 0; k < kActPieces; ++k) {
        uint16_t *to = s.act + ((int64_t)k * (j.tokens * j.top) + a) * s.ld_act + f;
        if (rows == 15) {
            *(uint2 *)to = uint2{(uint32_t)p[0][k] | (uint32_t)p[1][k] << 16, (uint32_t)p[2][k] | (uint32_t)p[3][k] << 16};
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (rows >> c & 1) to[c] = p[c][k];
        }
    }
}

template <int TYPE, int KS, int WK, bool FEW, bool FOLD>
__global__ __launch_bounds__(kThinThreads, two_on_a_cu(register_pieces(TYPE, FOLD), KS, FEW) ? 4 : 2) void up_kernel(StreamArgs args) {
    typedef typename MxType<TYPE>::T T;
    constexpr int G = group_of(register_pieces(TYPE, FOLD), KS, FEW);
    typedef MxTokens<TYPE, mx_pieces(TYPE), KS, WK, 1, FOLD> Tokens;
    typedef MxStream<2, G, KS, WK, true> Stream;
    const MxMoeJob &j = args.j;
    const Scratch &s = args.s;
    const MxWeights &w = args.w;
    // red, then the sums kept from one piece of K to the next.
    extern __shared__ __attribute__((aligned(16))) f32v4 red[];
    __shared__ std::conditional_t<FEW, Choice, Listed> choice;
    const int lane = threadIdx.x & 63, kw = (threadIdx.x >> 6) % WK;
    Tokens x;
    Stream stream;
    const int tiles = up_tiles(j), first = blockIdx.x * args.per, end = first + args.per < tiles ? first + args.per : tiles;
    int e = blockIdx.y, n = 1;
    const auto row_of = [&](int tile, int m) { return up_row(j, e, tile, m); };
    if constexpr (FEW) {
        // blockIdx.y: a choice.  Its token is known before its expert.
        const int t = blockIdx.y / j.top;
        const T *row[1] = {x.token() == 0 ? (const T *)j.x + (int64_t)t * j.ldx : nullptr};
        x.load(row, kw * KS, j.hidden, lane >> 4);
        rank_experts(j, s.logits + (int64_t)t * j.experts, choice);
        e = choice.expert[blockIdx.y % j.top];
    } else {
        n = list_tokens(j, s.chosen, e, choice);
    }
    bool odd = false;
    for (int i0 = 0; i0 < n; i0 += x.kTokens) {
        const T *row[1] = {nullptr};
        if (x.token() >= 0 && i0 + x.token() < n) {
            int t;
            if constexpr (FEW) t = blockIdx.y / j.top;
            else t = choice.token[i0 + x.token()];
            row[0] = (const T *)j.x + (int64_t)t * j.ldx;
        }
        for (int s0 = 0; s0 < w.slabs; s0 += WK * KS) {
            if (!FEW || s0 > 0) x.load(row, s0 + kw * KS, j.hidden, lane >> 4);
            stream.begin(w, s0 + kw * KS, first, end, row_of);
            stream.run(x, w, s0 + kw * KS, first, end, red, red + kThinSums<G, 1>, s0 == 0, s0 + WK * KS >= w.slabs, odd, row_of,
                       [&](int tile, int, int l, const f32v4(&v)[2], int rows) {
                           const int i = i0 + (l & 15);
                           if (i >= n) return;
                           int a = blockIdx.y;
                           if constexpr (!FEW) a = choice.list[i];
                           store_activations(j, s, a, (tile >> 1) * 16 + 4 * (l >> 4), v[0], v[1], rows);
                       });
        }
    }
    if constexpr (FEW)
        if (blockIdx.x == 0 && blockIdx.y % j.top == 0) {
            const int t = blockIdx.y / j.top;
            write_choice(j, s, t, s.logits + (int64_t)t * j.experts, choice);
        }
    if (__builtin_expect(odd, 0)) {   // weights beyond the largest float?
        const StreamArgs b = mx_arguments<StreamArgs>();
        const int tiles = up_tiles(b.j), first = blockIdx.x * b.per, end = first + b.per < tiles ? first + b.per : tiles;
        int count = 1;
        if constexpr (!FEW) count = choice.count;
        const auto choice_of = [&](int i) {
            if constexpr (FEW) return (int)blockIdx.y;
            else return choice.list[i];
        };
        const auto token_of = [&](int i) {
            if constexpr (FEW) return (int)blockIdx.y / b.j.top;
            else return choice.token[i];
        };
        int e;
        if constexpr (FEW) e = choice.expert[blockIdx.y % b.j.top];
        else e = choice.expert;
#pragma nounroll
        for (int i0 = 0; i0 < count; i0 += Tokens::kTokens)
            Stream::template mend<1, Tokens::kTokens>(
                b.w, 0, b.w.slabs, first, end, [&](int tile, int m) { return up_row(b.j, e, tile, m); },
                [&](int, int t, int column) {
                    if (i0 + t >= count || column >= b.j.hidden) return 0.0f;
                    return MxType<TYPE>::load((const T *)b.j.x + (int64_t)token_of(i0 + t) * b.j.ldx + column);
                },
                [&](int tile, int, int l, const f32v4(&v)[2], int rows) {
                    const int i = i0 + (l & 15);
                    if (i < count) store_activations(b.j, b.s, choice_of(i), (tile >> 1) * 16 + 4 * (l >> 4), v[0], v[1], rows);
                });
    }
}

// ---- down ----

// An inner activation of choice a from its pieces, zero beyond the last.
__device__ __forceinline__ float activation(const MxMoeJob &j, const Scratch &s, int a, int column) {
    if (column >= j.inner) return 0.0f;
    float v = 0.0f;
#pragma unroll
    for (int p = 0; p < kActPieces; ++p)
        v += MxType<SGEMM_TYPE_BF16>::load(s.act + ((int64_t)p * (j.tokens * j.top) + a) * s.ld_act + column);
    return v;
}

__device__ __forceinline__ int64_t down_row(const MxMoeJob &j, int e, int tile, int m) {
    const int h = tile * 16 + m;
    return (int64_t)e * j.hidden + (h < j.hidden ? h : j.hidden - 1);
}

template <int KS, int WK, bool FOLD>
__global__ __launch_bounds__(kThinThreads, two_on_a_cu(FOLD ? 1 : kActPieces, KS, false) ? 4 : 2) void down_kernel(StreamArgs args) {
    constexpr int G = group_of(FOLD ? 1 : kActPieces, KS, false);
    typedef MxTokens<SGEMM_TYPE_BF16, kActPieces, KS, WK, 1, FOLD> Tokens;
    typedef MxStream<1, G, KS, WK, true> Stream;
    const MxMoeJob &j = args.j;
    const Scratch &s = args.s;
    const MxWeights &w = args.w;
    Tokens x;
    extern __shared__ __attribute__((aligned(16))) f32v4 red[];
    __shared__ Listed choice;
    const int lane = threadIdx.x & 63, kw = (threadIdx.x >> 6) % WK;
    int e;
    const int n = list_tokens(j, s.chosen, e, choice);
    const int *list = choice.list;
    const int tiles = (j.hidden + 15) / 16, first = blockIdx.x * args.per, end = first + args.per < tiles ? first + args.per : tiles;
    const auto row_of = [&](int tile, int m) { return down_row(j, e, tile, m); };
    Stream stream;
    bool odd = false;
    for (int i0 = 0; i0 < n; i0 += x.kTokens) {
        const int t = x.token();
        const uint16_t *row = t >= 0 && i0 + t < n ? s.act + (int64_t)list[i0 + t] * s.ld_act : nullptr;
        for (int s0 = 0; s0 < w.slabs; s0 += WK * KS) {
            x.load_pieces(row, (int64_t)j.tokens * j.top * s.ld_act, s0 + kw * KS, (int)s.ld_act, lane >> 4);
            stream.begin(w, s0 + kw * KS, first, end, row_of);
            stream.run(x, w, s0 + kw * KS, first, end, red, red + kThinSums<G, 1>, s0 == 0, s0 + WK * KS >= w.slabs, odd, row_of,
                       [&](int tile, int, int l, const f32v4(&v)[1], int rows) {
                           const int i = i0 + (l & 15);
                           if (i < n) mx_store_rows(s.part + (int64_t)list[i] * s.ld_part + tile * 16 + 4 * (l >> 4), v[0], rows);
                       });
        }
    }
    if (__builtin_expect(odd, 0)) {   // weights beyond the largest float?
        const StreamArgs b = mx_arguments<StreamArgs>();
        const int tiles = (b.j.hidden + 15) / 16, first = blockIdx.x * b.per, end = first + b.per < tiles ? first + b.per : tiles;
#pragma nounroll
        for (int i0 = 0; i0 < choice.count; i0 += Tokens::kTokens)
            Stream::template mend<1, Tokens::kTokens>(
                b.w, 0, b.w.slabs, first, end, [&](int tile, int m) { return down_row(b.j, choice.expert, tile, m); },
                [&](int, int t, int column) { return i0 + t < choice.count ? activation(b.j, b.s, choice.list[i0 + t], column) : 0.0f; },
                [&](int tile, int, int l, const f32v4(&v)[1], int rows) {
                    const int i = i0 + (l & 15);
                    if (i < choice.count)
                        mx_store_rows(b.s.part + (int64_t)choice.list[i] * b.s.ld_part + tile * 16 + 4 * (l >> 4), v[0], rows);
                });
    }
}

template <int TYPE>
__global__ __launch_bounds__(256) void join_kernel(MxMoeJob j, Scratch s) {
    const int h = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (h >= j.hidden) return;
    float sum = 0.0f;
#pragma unroll 8
    for (int i = t * j.top; i < (t + 1) * j.top; ++i) sum = fmaf(s.weight[i], s.part[i * s.ld_part + h], sum);
    ((typename MxType<TYPE>::T *)j.y)[t * j.ldy + h] = MxType<TYPE>::from(sum);
}

template <int TYPE>
__global__ __launch_bounds__(kThinThreads) void down_few_kernel(MxMoeJob j, Scratch s, MxWeights w) {
    typedef typename MxType<TYPE>::T T;
    constexpr int P = kActPieces, U = 6;
    __shared__ float ys[kThinWaves][kFew][16];   // a wave's sums: token, row
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, q = lane >> 4;
    const int all = j.tokens * j.top, h0 = blockIdx.x * 16;
    const int h = h0 + l16 < j.hidden ? h0 + l16 : j.hidden - 1;
    for (int i = lane; i < kFew * 16; i += 64) (&ys[wave][0][0])[i] = 0.0f;
    // This wave's part of the (choice, slab) list.
    const int64_t items = (int64_t)all * w.slabs;
    int64_t at = items * wave / kThinWaves;
    const int64_t stop = items * (wave + 1) / kThinWaves;
    while (at < stop) {
        const int a = (int)(at / w.slabs), s_begin = (int)(at - (int64_t)a * w.slabs);
        const int s_end = stop - at < w.slabs - s_begin ? s_begin + (int)(stop - at) : w.slabs;
        at += s_end - s_begin;
        const int64_t r = (int64_t)s.chosen[a] * j.hidden + h;
        const float weight = s.weight[a];
        const uint16_t *act = s.act + a * s.ld_act;
        f32v4 acc{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s0 = s_begin; s0 < s_end; s0 += U) {
            MxBlock b[U];
            uint4 x[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) b[u] = s0 + u < s_end ? w.load(r, s0 + u, q) : MxBlock{uint4{0, 0, 0, 0}, 0};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // one token, folded: piece p in column p
                    const int c = (s0 + u) * kMxSlab + 32 * q + 8 * k;
                    x[u][k] = l16 < P && s0 + u < s_end && c < s.ld_act ? *(const uint4 *)(act + l16 * all * s.ld_act + c)
                                                                        : uint4{0, 0, 0, 0};
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t c[4] = {b[u].codes.x, b[u].codes.y, b[u].codes.z, b[u].codes.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) acc = mx_mfma(mx_bf16x8(c[k], mx_scale(b[u], q)), x[u][k], acc);
            }
        }
        f32v4 sum = acc;
#pragma unroll
        for (int p = 1; p < P; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k) sum[k] += __shfl(acc[k], (lane & 48) + p, 64);
        if (l16 == 0) {
            f32v4 *y = (f32v4 *)&ys[wave][a / j.top][4 * q];
            *y += weight * sum;
        }
    }
    __syncthreads();
    static_assert(kFew * 16 <= kThinThreads, "a thread takes one result");
    const int t = tid >> 4, r = tid & 15;
    const bool mine = t < j.tokens && h0 + r < j.hidden;
    float sum = 0.0f;
    if (mine) {
        sum = ys[0][t][r];
#pragma unroll
        for (int k = 1; k < kThinWaves; ++k) sum += ys[k][t][r];
        ((T *)j.y)[t * j.ldy + h0 + r] = MxType<TYPE>::from(sum);
    }
    // Once more those to which a weight beyond the largest float adds.
    for (uint64_t odd = __ballot(mine && !mx_finite(sum)); __builtin_expect(odd != 0, 0); odd &= odd - 1) {
        const int l = __ffsll((unsigned long long)odd) - 1, i = __builtin_amdgcn_readfirstlane(wave) * 64 + l;
        const int begin = (i >> 4) * j.top, end = begin + j.top;
        const auto row = [&](int a) { return (int64_t)s.chosen[a] * j.hidden + h0 + (i & 15); };
        bool beyond = false;
#pragma nounroll
        for (int a = begin; a < end; ++a) beyond |= mx_beyond(w, row(a), 0, w.slabs);
        if (!beyond) continue;
        sum = 0.0f;
#pragma nounroll
        for (int a = begin; a < end; ++a)
            sum = fmaf(s.weight[a], mx_plain_sum(w, row(a), 0, w.slabs, [&](int column) { return activation(j, s, a, column); }), sum);
        if (lane == l) ((T *)j.y)[t * j.ldy + h0 + r] = MxType<TYPE>::from(sum);
    }
}

// ---- launches ----

// Workgroups along the rows: enough that `slots` times as many are `fill`, and
// not more tiles each than `most`.
int groups_of(int tiles, int unit, int slots, int fill, int most) {
    const int want = (fill + slots - 1) / slots, least = (tiles + most - 1) / most;
    const int groups = want > least ? want : least, units = (tiles + unit - 1) / unit;
    return groups < units ? groups : units;
}

// LDS of a streaming kernel, and the most tiles a workgroup takes, when K
// comes in several pieces (their sums stay in LDS).
constexpr int kCarryTiles = 32;

template <int TYPE, int KS, int WK, bool FEW, bool FOLD>
hipError_t launch_up(MxMoeJob &j, Scratch &s, hipStream_t stream) {
    constexpr int P = register_pieces(TYPE, FOLD), G = group_of(P, KS, FEW);
    StreamArgs args{j, s, mx_weights(j.up, j.sup, (int64_t)2 * j.experts * j.inner, j.hidden), 0};
    const int tiles = up_tiles(j), all = j.tokens * j.top, slots = FEW ? all : expert_rows(j);
    const bool pieces = args.w.slabs > WK * KS;
    const int fill = FEW && !two_on_a_cu(P, KS, FEW) ? 256 : 512;
    const int per = args.per = mx_share(tiles, groups_of(tiles, 2, slots, fill, pieces ? kCarryTiles : tiles), 2);
    const int bytes = (kThinSums<G, 1> + (pieces ? kCarryTiles * 64 : 0)) * 16;
    void *params[] = {&args};
    return hipLaunchKernel((const void *)up_kernel<TYPE, KS, WK, FEW, FOLD>,
                           dim3((unsigned)((tiles + per - 1) / per), (unsigned)slots), dim3(kThinThreads), params, bytes, stream);
}

// (slabs a wave keeps, waves along K) for a number of slabs.  Where K is short,
// so few waves share it that none idles; else eight waves take two slabs each,
// several runs of them if need be.  The layer for 32 tokens, 8 of 64 experts, in
// us, against eight waves of two slabs for every length:
//   hidden (inner 768)    256         512         1024
//   bf16                  24.8 / 34.5 29.7 / 36.9 36.5 / 41.1
//   fp16                  27.7 / 49.6 31.9 / 52.9 40.2 / 57.4
//   fp32                  27.7 / 49.1 31.8 / 53.6 46.5 / 57.4
// (Two pieces of two slabs have a CU to themselves: fp16, 768 x 512: 43.2 with
// two slabs, 36.2 with one.)  bf16 beyond 24 slabs goes by whole runs of four
// (24 tokens, 8 of 128 experts, 4096 x 1536: 250 against 271 us; 8 tokens, 6144 x
// 1024: 143 against 129; 64 tokens, 4096 x 1024: the same).  Few choices: latency
// counts, all waves along K.
template <int TYPE, bool FEW, bool FOLD>
hipError_t launch_up_slabs(MxMoeJob &j, Scratch &s, hipStream_t stream) {
    constexpr int P = register_pieces(TYPE, FOLD);
    const int n = mx_slabs(j.hidden);
    if constexpr (FEW) {
        if (n <= 8) return launch_up<TYPE, 1, 8, FEW, FOLD>(j, s, stream);
        if constexpr (P == 1)
            if (n > 16) return launch_up<TYPE, 4, 8, FEW, FOLD>(j, s, stream);
    } else {
        if (n <= 2) return launch_up<TYPE, 1, 2, FEW, FOLD>(j, s, stream);
        if (n <= 4) return launch_up<TYPE, 1, 4, FEW, FOLD>(j, s, stream);
        if (n <= 8) return launch_up<TYPE, P == 2 ? 1 : 2, P == 2 ? 8 : 4, FEW, FOLD>(j, s, stream);
        if constexpr (P == 1 && !FOLD)
            if (n > 24) return launch_up<TYPE, 4, 8, FEW, FOLD>(j, s, stream);
    }
    return launch_up<TYPE, 2, 8, FEW, FOLD>(j, s, stream);
}

template <int KS, int WK, bool FOLD>
hipError_t launch_down(MxMoeJob &j, Scratch &s, hipStream_t stream) {
    StreamArgs args{j, s, mx_weights(j.down, j.sdown, (int64_t)j.experts * j.hidden, j.inner), 0};
    const int tiles = (j.hidden + 15) / 16, slots = expert_rows(j);
    const bool pieces = args.w.slabs > WK * KS;
    const int per = args.per = mx_share(tiles, groups_of(tiles, 1, slots, 512, pieces ? kCarryTiles : tiles), 1);
    const int bytes = (kThinSums<group_of(FOLD ? 1 : kActPieces, KS, false), 1> + (pieces ? kCarryTiles * 64 : 0)) * 16;
    void *params[] = {&args};
    return hipLaunchKernel((const void *)down_kernel<KS, WK, FOLD>, dim3((unsigned)((tiles + per - 1) / per), (unsigned)slots),
                           dim3(kThinThreads), params, bytes, stream);
}

// The same.  Unfolded, three pieces of more than one slab take a CU to themselves:
// beyond two slabs K goes in runs of eight past two workgroups on a CU (48 tokens, 8
// of 128 experts, 4096 x 1536 bf16: 265 us so, 278 with two slabs a wave; 20 tokens,
// 2 of 16, 4096 x 4096: 106 against 114; 32 tokens, 8 of 64, 2048 x 512: 43.5 against
// 45.7).  Folded, against eight waves of three slabs for every length, 4 tokens, 8 of
// 64 experts of hidden 2048: inner 128 19.6 / 30.7 us, 256 21.8 / 32.2, 512 25.9 /
// 35.6, 768 35.4 / 38.5, 1024 34.9 / 41.2, 2048 56.0 / 59.6, 4096 90.9 / 100.8.
template <bool FOLD>
hipError_t launch_down_slabs(MxMoeJob &j, Scratch &s, hipStream_t stream) {
    const int n = mx_slabs(j.inner);
    if (n <= 1) return launch_down<1, 1, FOLD>(j, s, stream);
    if (n <= 2) return launch_down<1, 2, FOLD>(j, s, stream);
    if constexpr (FOLD) {
        if (n <= 4) return launch_down<2, 2, FOLD>(j, s, stream);
        if (n <= 6) return launch_down<3, 2, FOLD>(j, s, stream);
        if (n <= 8) return launch_down<2, 4, FOLD>(j, s, stream);
        if (n <= 16) return launch_down<4, 4, FOLD>(j, s, stream);
        return n > 24 ? launch_down<4, 8, FOLD>(j, s, stream) : launch_down<3, 8, FOLD>(j, s, stream);
    } else {
        return launch_down<1, 8, FOLD>(j, s, stream);
    }
}

// Whether an expert's tokens always fit a folded tile.  (Where only most do, the
// few workgroups that stream their weights twice are what the kernel waits for:
// `down` of two pieces, 48 tokens, 8 of 128 experts, 4096 x 1536: 124 us, unfolded 104.)
bool folds(const MxMoeJob &j, int pieces) { return j.tokens <= 16 / pieces; }

template <int TYPE>
hipError_t launch_type(const MxMoeJob &job, hipStream_t stream) {
    MxMoeJob j = job;
    Scratch s = layout(j.scratch, j.tokens, j.hidden, j.inner, j.experts, j.top);
    void *params[] = {&j, &s};
    const unsigned ge = (unsigned)((j.experts + 3) / 4);
    hipError_t e = j.tokens < 4 ? hipLaunchKernel((const void *)logits_kernel<TYPE, 1>, dim3(ge, (unsigned)j.tokens), dim3(256),
                                                  params, 0, stream)
                                : hipLaunchKernel((const void *)logits_kernel<TYPE, 4>, dim3(ge, (unsigned)((j.tokens + 3) / 4)),
                                                  dim3(256), params, 0, stream);
    if (e != hipSuccess) return e;
    if (j.tokens * j.top <= kFew) {
        e = launch_up_slabs<TYPE, true, (mx_pieces(TYPE) > 1)>(j, s, stream);
        if (e != hipSuccess) return e;
        MxWeights w = mx_weights(j.down, j.sdown, (int64_t)j.experts * j.hidden, j.inner);
        void *down[] = {&j, &s, &w};
        return hipLaunchKernel((const void *)down_few_kernel<TYPE>, dim3((unsigned)((j.hidden + 15) / 16)), dim3(kThinThreads), down,
                               0, stream);
    }
    e = hipLaunchKernel((const void *)choose_kernel, dim3((unsigned)j.tokens), dim3(kThinThreads), params, 0, stream);
    if (e != hipSuccess) return e;
    constexpr int PX = mx_pieces(TYPE);
    if (PX > 1 && folds(j, PX)) e = launch_up_slabs<TYPE, false, (PX > 1)>(j, s, stream);
    else e = launch_up_slabs<TYPE, false, false>(j, s, stream);
    if (e != hipSuccess) return e;
    e = folds(j, kActPieces) ? launch_down_slabs<true>(j, s, stream) : launch_down_slabs<false>(j, s, stream);
    if (e != hipSuccess) return e;
    return hipLaunchKernel((const void *)join_kernel<TYPE>, dim3((unsigned)((j.hidden + 255) / 256), (unsigned)j.tokens), dim3(256),
                           params, 0, stream);
}

}  // namespace

int64_t mx4_moe_scratch(int tokens, int hidden, int inner, int experts, int top) {
    return layout(nullptr, tokens, hidden, inner, experts, top).bytes;
}

hipError_t launch_mx4_moe(const MxMoeJob &j, hipStream_t s) {
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_type<SGEMM_TYPE_F32>(j, s);
    case SGEMM_TYPE_BF16: return launch_type<SGEMM_TYPE_BF16>(j, s);
    case SGEMM_TYPE_F16: return launch_type<SGEMM_TYPE_F16>(j, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace sgemm
