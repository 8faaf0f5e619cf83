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
// Bound by reading the chosen experts once: 3 F H 0.53 bytes each.  Three
// kernels:
//   route   logits in 64 bits (which expert is chosen must not hang on the
//           order of a sum), the tokens as bf16 pieces, and, by the last
//           workgroup of a group of tokens to arrive, choice and weights
//   up      a workgroup takes 16 inner columns of one expert: their gate and
//           up rows, all tokens of the expert; writes silu(g) * u, again as
//           bf16 pieces
//   down    a workgroup takes 16 rows of the output and every expert: its
//           waves share the (expert, slab) list evenly and add p_e times
//           their part into sums of their own, which are added in wave order
// Every sum has a fixed order: results repeat bit for bit.  Activations are
// held to 24 bits (three pieces) for fp32 outputs and to 16 (two) for 16-bit
// ones, whose own rounding is at least 32 times coarser.
#include "mx4_thin.h"

namespace sgemm {
namespace {

constexpr int kWaves = 8;
constexpr int act_pieces(int type) { return type == SGEMM_TYPE_F32 ? 3 : 2; }

// Scratch memory, every part 256-byte aligned.
struct Scratch {
    double *logits;      // tokens x experts
    int *chosen;         // tokens x top
    float *weight;       // tokens x top
    uint16_t *x;         // pieces x tokens x hp
    uint16_t *act;       // pieces x (tokens * top) x fp
    int64_t bytes;
};

inline __host__ __device__ int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

Scratch layout(char *p, int tokens, int hidden, int inner, int experts, int top, int type) {
    Scratch s;
    int64_t at = 0;
    const auto take = [&](int64_t n) { const int64_t here = at; at += up256(n); return p + here; };
    s.logits = (double *)take((int64_t)tokens * experts * 8);
    s.chosen = (int *)take((int64_t)tokens * top * 4);
    s.weight = (float *)take((int64_t)tokens * top * 4);
    s.x = (uint16_t *)take((int64_t)mx_pieces(type) * tokens * mx_slabs(hidden) * kMxSlab * 2);
    s.act = (uint16_t *)take((int64_t)act_pieces(type) * tokens * top * mx_slabs(inner) * kMxSlab * 2);
    s.bytes = at;
    return s;
}

// ---- route ----

template <int TYPE, int TT>
__global__ __launch_bounds__(256) void logits_kernel(MxMoeJob j, Scratch s, int vec) {
    typedef typename MxType<TYPE>::T T;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 4 + wave, t0 = blockIdx.y * TT;
    const int hp = mx_slabs(j.hidden) * kMxSlab;
    const T *r = (const T *)j.router + (e < j.experts ? e : 0) * j.ldr;
    const T *x[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t] = (const T *)j.x + (t0 + t < j.tokens ? t0 + t : t0) * j.ldx;
    double sum[TT] = {};
    for (int h = 8 * lane; h < j.hidden; h += 512) {
        float w[8], v[8];
        mx_load_edge8<TYPE>(r, h, j.hidden, vec, w);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            mx_load_edge8<TYPE>(x[t], h, j.hidden, vec, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[t] = fma((double)w[i], (double)v[i], sum[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum[t] += __shfl_xor(sum[t], off, 64);
        if (lane == 0 && e < j.experts && t0 + t < j.tokens) s.logits[(t0 + t) * j.experts + e] = sum[t];
    }
    // The tokens as pieces, zeros up to whole slabs; the group's workgroups share the columns.
    constexpr int P = mx_pieces(TYPE);
    for (int h = blockIdx.x * 256 + threadIdx.x; h < hp; h += gridDim.x * 256)
        for (int t = 0; t < TT && t0 + t < j.tokens; ++t) {
            uint16_t p[P];
            const T *row = (const T *)j.x + (t0 + t) * j.ldx;
            mx_split<P>(h < j.hidden ? MxType<TYPE>::load(row + h) : 0.0f, p);
#pragma unroll
            for (int i = 0; i < P; ++i) s.x[((int64_t)i * j.tokens + t0 + t) * hp + h] = p[i];
        }
}

// A logit as an integer of the same order: NaN above all, -0 equal to 0.
__device__ __forceinline__ int64_t order_key(double v) {
    if (v != v) return INT64_MAX;
    const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
    return b < 0 ? b ^ INT64_MAX : b;
}

// One workgroup per token: an expert's rank is the number of experts before it.
__global__ __launch_bounds__(256) void choose_kernel(MxMoeJob j, Scratch s) {
    __shared__ int64_t key[SGEMM_MX4_MAX_EXPERTS];
    __shared__ float ex[SGEMM_MX4_MAX_EXPERTS];
    __shared__ double best;
    __shared__ float part[4];
    __shared__ float picked[SGEMM_MX4_MAX_TOP];
    const int t = blockIdx.x, tid = threadIdx.x;
    const double *l = s.logits + (int64_t)t * j.experts;
    for (int e = tid; e < j.experts; e += 256) key[e] = order_key(l[e]);
    __syncthreads();
    int rank[SGEMM_MX4_MAX_EXPERTS / 256];
#pragma unroll
    for (int i = 0; i < SGEMM_MX4_MAX_EXPERTS / 256; ++i) {
        const int e = tid + 256 * i;
        rank[i] = 0;
        if (e >= j.experts) continue;
        const int64_t mine = key[e];
        int n = 0;
        for (int o = 0; o < j.experts; ++o) n += key[o] > mine || (key[o] == mine && o < e);
        rank[i] = n;
        if (n == 0) best = l[e];
    }
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < SGEMM_MX4_MAX_EXPERTS / 256; ++i) {
        const int e = tid + 256 * i;
        if (e >= j.experts) continue;
        const float v = expf((float)(l[e] - best));
        total += v;
        if (rank[i] < j.top) {
            picked[rank[i]] = v;
            s.chosen[t * j.top + rank[i]] = e;
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) total += __shfl_xor(total, off, 64);
    if ((tid & 63) == 0) part[tid >> 6] = total;
    __syncthreads();
    if (tid < j.top) {
        float sum = 0.0f;
        if (j.norm)
            for (int i = 0; i < j.top; ++i) sum += picked[i];
        else
            sum = ((part[0] + part[1]) + part[2]) + part[3];
        s.weight[t * j.top + tid] = picked[tid] / sum;
    }
}

// ---- up ----

template <int TYPE, int MT>
__global__ __launch_bounds__(64 * kWaves) void up_kernel(MxMoeJob j, Scratch s) {
    constexpr int P = mx_pieces(TYPE), PA = act_pieces(TYPE), U = 2;
    __shared__ __attribute__((aligned(16))) f32v4 red[kWaves * 2 * MT * 64];
    __shared__ int list[SGEMM_MX4_MAX_TOKENS];
    __shared__ int count, earlier;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int all = j.tokens * j.top, f0 = blockIdx.x * 16;
    // blockIdx.y: an expert, or, with fewer choices than experts, a choice,
    // which stands for its expert if none before it does.
    const bool by_choice = all < j.experts;
    const int e = by_choice ? s.chosen[blockIdx.y] : blockIdx.y;
    if (tid == 0) count = 0, earlier = 0;
    __syncthreads();
    for (int a = tid; a < all; a += 64 * kWaves)
        if (s.chosen[a] == e) {
            list[atomicAdd(&count, 1)] = a;   // any order: a token's result does not depend on its place
            if (by_choice && a < (int)blockIdx.y) earlier = 1;
        }
    __syncthreads();
    const int n = count;
    if (n == 0 || earlier) return;

    const int slabs = mx_slabs(j.hidden), hp = slabs * kMxSlab, fp = mx_slabs(j.inner) * kMxSlab;
    const int64_t rows = (int64_t)2 * j.experts * j.inner, plane = mx_plane_rows(rows);
    const int l16 = lane & 15, q = lane >> 4;
    const int f = f0 + l16 < j.inner ? f0 + l16 : j.inner - 1;
    const int64_t rg = (int64_t)2 * e * j.inner + f, ru = rg + j.inner;
    const int64_t rowb = (int64_t)slabs * kMxSlabBytes;
    const uint16_t *x[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int i = mt * 16 + l16 < n ? mt * 16 + l16 : n - 1;
        x[mt] = s.x + (int64_t)(list[i] / j.top) * hp + 32 * q;
    }
    f32v4 acc[2][MT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[r][mt] = f32v4{0.0f, 0.0f, 0.0f, 0.0f};
    if (f0 < j.inner)
        for (int s0 = wave; s0 < slabs; s0 += kWaves * U) {
            MxBlock b[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int slab = s0 + kWaves * u;
                b[u][0] = mx_block(j.up + rg * rowb, (const uint32_t *)j.sup + rg, plane, slab, q, slab < slabs);
                b[u][1] = mx_block(j.up + ru * rowb, (const uint32_t *)j.sup + ru, plane, slab, q, slab < slabs);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int slab = s0 + kWaves * u;
                if (slab >= slabs) break;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if (mt * 16 >= n) break;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint4 xs[P];
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            xs[p] = *(const uint4 *)(x[mt] + (int64_t)p * j.tokens * hp + slab * kMxSlab + 8 * k);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint4 c = b[u][r].codes;
                            const bf16v8 w = mx_bf16x8(k == 0 ? c.x : k == 1 ? c.y : k == 2 ? c.z : c.w, mx_scale(b[u][r], q));
#pragma unroll
                            for (int p = 0; p < P; ++p) acc[r][mt] = mx_mfma(w, xs[p], acc[r][mt]);
                        }
                    }
                }
            }
        }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) red[((wave * 2 + r) * MT + mt) * 64 + lane] = acc[r][mt];
    __syncthreads();
    for (int i = tid; i < MT * 64; i += 64 * kWaves) {
        const int l = i & 63, mt = i >> 6, t = mt * 16 + (l & 15);
        if (t >= n) continue;
        f32v4 g = red[i], u = red[MT * 64 + i];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) g += red[w * (2 * MT * 64) + i], u += red[(w * 2 + 1) * MT * 64 + i];
        const int fc = f0 + 4 * (l >> 4);
        uint16_t p[4][PA];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            mx_split<PA>(fc + c < j.inner ? g[c] / (1.0f + expf(-g[c])) * u[c] : 0.0f, p[c]);
#pragma unroll
        for (int k = 0; k < PA; ++k)
            *(uint2 *)(s.act + ((int64_t)k * all + list[t]) * fp + fc) =
                uint2{(uint32_t)p[0][k] | (uint32_t)p[1][k] << 16, (uint32_t)p[2][k] | (uint32_t)p[3][k] << 16};
    }
}

// ---- down ----

template <int TYPE, int MT>
__global__ __launch_bounds__(64 * kWaves) void down_kernel(MxMoeJob j, Scratch s) {
    typedef typename MxType<TYPE>::T T;
    constexpr int PA = act_pieces(TYPE), U = 4;
    __shared__ __attribute__((aligned(16))) float ys[kWaves * 16 * MT * 16];   // a wave's sums: token, row
    __shared__ int first[SGEMM_MX4_MAX_EXPERTS + 1], place[SGEMM_MX4_MAX_EXPERTS], active[SGEMM_MX4_MAX_EXPERTS];
    __shared__ uint16_t list[SGEMM_MX4_MAX_TOKENS * SGEMM_MX4_MAX_TOP];
    __shared__ int n_active;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int all = j.tokens * j.top;
    // The choices sorted by expert, and the experts that have any.
    for (int e = tid; e < j.experts; e += 64 * kWaves) place[e] = 0;
    for (int i = tid; i < kWaves * 16 * MT * 16; i += 64 * kWaves) ys[i] = 0.0f;
    __syncthreads();
    for (int a = tid; a < all; a += 64 * kWaves) atomicAdd(&place[s.chosen[a]], 1);
    __syncthreads();
    if (wave == 0) {
        int sum = 0, act = 0;
        for (int e0 = 0; e0 < j.experts; e0 += 64) {
            const int e = e0 + lane, c = e < j.experts ? place[e] : 0;
            int run = c;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int v = __shfl_up(run, off, 64);
                if (lane >= off) run += v;
            }
            const uint64_t some = __ballot(c > 0);
            if (e < j.experts) first[e] = sum + run - c;
            if (c > 0) active[act + __popcll(some & ((1ull << lane) - 1))] = e;
            sum += __shfl(run, 63, 64);
            act += __popcll(some);
        }
        if (lane == 0) first[j.experts] = sum, n_active = act;
    }
    __syncthreads();
    for (int e = tid; e < j.experts; e += 64 * kWaves) place[e] = first[e];
    __syncthreads();
    for (int a = tid; a < all; a += 64 * kWaves) list[atomicAdd(&place[s.chosen[a]], 1)] = (uint16_t)a;
    __syncthreads();

    const int slabs = mx_slabs(j.inner), fp = slabs * kMxSlab;
    const int64_t plane = mx_plane_rows((int64_t)j.experts * j.hidden), rowb = (int64_t)slabs * kMxSlabBytes;
    const int l16 = lane & 15, q = lane >> 4, h0 = blockIdx.x * 16;
    const int h = h0 + l16 < j.hidden ? h0 + l16 : j.hidden - 1;
    float *mine = ys + wave * (16 * MT * 16);
    // This wave's part of the (active expert, slab) list.
    const int64_t items = (int64_t)n_active * slabs;
    int64_t at = items * wave / kWaves;
    const int64_t end = items * (wave + 1) / kWaves;
    while (at < end) {
        const int i = (int)(at / slabs), s_begin = (int)(at - (int64_t)i * slabs);
        const int s_end = end - at < slabs - s_begin ? s_begin + (int)(end - at) : slabs;
        at += s_end - s_begin;
        const int e = active[i], from = first[e], n = first[e + 1] - from;
        const int64_t r = (int64_t)e * j.hidden + h;
        const uint8_t *row = j.down + r * rowb;
        const uint32_t *words = (const uint32_t *)j.sdown + r;
        const uint16_t *x[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int k = mt * 16 + l16 < n ? mt * 16 + l16 : n - 1;
            x[mt] = s.act + (int64_t)list[from + k] * fp + 32 * q;
        }
        f32v4 acc[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[mt] = f32v4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s0 = s_begin; s0 < s_end; s0 += U) {
            MxBlock b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) b[u] = mx_block(row, words, plane, s0 + u, q, s0 + u < s_end);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s0 + u >= s_end) break;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if (mt * 16 >= n) break;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 c = b[u].codes;
                        const bf16v8 w = mx_bf16x8(k == 0 ? c.x : k == 1 ? c.y : k == 2 ? c.z : c.w, mx_scale(b[u], q));
#pragma unroll
                        for (int p = 0; p < PA; ++p) {
                            const uint4 xs = *(const uint4 *)(x[mt] + (int64_t)p * all * fp + (s0 + u) * kMxSlab + 8 * k);
                            acc[mt] = mx_mfma(w, xs, acc[mt]);
                        }
                    }
                }
            }
        }
        // Lane l: rows 4 (l / 16) .. + 3 for the expert's token l % 16.
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int k = mt * 16 + l16;
            if (k < n) {
                const int a = list[from + k];
                const float p = s.weight[a];
                f32v4 *y = (f32v4 *)(mine + (a / j.top) * 16 + 4 * q);
                *y += p * acc[mt];
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < j.tokens * 16; i += 64 * kWaves) {
        const int t = i >> 4, r = i & 15;
        float sum = ys[i];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += ys[w * (16 * MT * 16) + i];
        if (h0 + r < j.hidden) ((T *)j.y)[t * j.ldy + h0 + r] = MxType<TYPE>::from(sum);
    }
}

template <int TYPE, int MT>
hipError_t launch_experts(MxMoeJob &j, Scratch &s, hipStream_t stream) {
    void *params[] = {&j, &s};
    const int all = j.tokens * j.top;
    hipError_t e = hipLaunchKernel((const void *)up_kernel<TYPE, MT>,
                                   dim3((unsigned)(mx_slabs(j.inner) * kMxSlab / 16), (unsigned)(all < j.experts ? all : j.experts)),
                                   dim3(64 * kWaves), params, 0, stream);
    if (e != hipSuccess) return e;
    return hipLaunchKernel((const void *)down_kernel<TYPE, MT>, dim3((unsigned)((j.hidden + 15) / 16)), dim3(64 * kWaves),
                           params, 0, stream);
}

template <int TYPE>
hipError_t launch_type(const MxMoeJob &job, hipStream_t stream) {
    MxMoeJob j = job;
    Scratch s = layout(j.scratch, j.tokens, j.hidden, j.inner, j.experts, j.top, TYPE);
    const int64_t b = TYPE == SGEMM_TYPE_F32 ? 4 : 2;
    int vec = ((uintptr_t)j.x & 15) == 0 && ((uintptr_t)j.router & 15) == 0 && (j.ldx * b & 15) == 0 && (j.ldr * b & 15) == 0;
    void *params[] = {&j, &s, &vec};
    const unsigned ge = (unsigned)((j.experts + 3) / 4);
    hipError_t e = j.tokens < 4 ? hipLaunchKernel((const void *)logits_kernel<TYPE, 1>, dim3(ge, (unsigned)j.tokens), dim3(256),
                                                  params, 0, stream)
                                : hipLaunchKernel((const void *)logits_kernel<TYPE, 4>, dim3(ge, (unsigned)((j.tokens + 3) / 4)),
                                                  dim3(256), params, 0, stream);
    if (e != hipSuccess) return e;
    e = hipLaunchKernel((const void *)choose_kernel, dim3((unsigned)j.tokens), dim3(256), params, 0, stream);
    if (e != hipSuccess) return e;
    if (j.tokens <= 16) return launch_experts<TYPE, 1>(j, s, stream);
    if (j.tokens <= 32) return launch_experts<TYPE, 2>(j, s, stream);
    return launch_experts<TYPE, 4>(j, s, stream);
}

}  // namespace

int64_t mx4_moe_scratch(int tokens, int hidden, int inner, int experts, int top, int type) {
    return layout(nullptr, tokens, hidden, inner, experts, top, type).bytes;
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
