// Y = X W^T for a few rows X of floats and 4-bit weights W (N x K): the
// product of single tokens, bound by reading W once (0.53 bytes a weight).
//
// A workgroup takes 16 R rows of W and up to 16 MT tokens; its 8 waves split
// K slab by slab (neighbouring waves read neighbouring 64-byte pieces of the
// same rows), each with U slabs of weights in flight, and their sums are
// added in wave order through LDS: no partials in memory, the same bits every
// time.  More tokens than 64 take further workgroups (blockIdx.y), which
// find the weights in the caches.
//
// bf16 tokens whose rows start on 16-byte boundaries are loaded straight into
// operand registers.  Other types and layouts go through LDS: a wave splits
// its own slab of the tokens into bf16 pieces there, loaded one step ahead.
#include "mx4_thin.h"

namespace sgemm {
namespace {

constexpr int kWaves = 8;
constexpr int kPieceRow = 272;   // bytes of a token's 128 pieces in LDS: 16 more than they take, against bank conflicts

template <int TYPE, bool STAGE, int R, int MT>
__global__ __launch_bounds__(64 * kWaves) void linear_kernel(MxLinearJob j, int vec) {
    typedef typename MxType<TYPE>::T T;
    constexpr int P = mx_pieces(TYPE), U = 4;
    static_assert(STAGE || P == 1, "one piece without staging");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n0 = blockIdx.x * 16 * R, m0 = blockIdx.y * 16 * MT;
    const int slabs = mx_slabs(j.K);
    const int64_t plane = mx_plane_rows(j.N);
    const int l16 = lane & 15, q = lane >> 4;
    const int tokens = j.M - m0 < 16 * MT ? j.M - m0 : 16 * MT;

    const uint8_t *row[R];
    const uint32_t *words[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = n0 + 16 * r + l16 < j.N ? n0 + 16 * r + l16 : j.N - 1;   // rows past N: computed, not stored
        row[r] = j.codes + n * ((int64_t)slabs * kMxSlabBytes);
        words[r] = (const uint32_t *)j.scales + n;
    }
    const T *x = (const T *)j.x + m0 * j.ldx;

    // Direct operands: token l16 of tile mt, columns of step s.
    auto direct = [&](int mt, int k) -> uint4 {
        if constexpr (!STAGE) {
            const int t = mt * 16 + l16;
            if (t < tokens) {
                const T *p = x + t * j.ldx + k;
                if (k + 8 <= j.K) return *(const uint4 *)p;
                uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + i < j.K) u[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
                return uint4{u[0], u[1], u[2], u[3]};
            }
        }
        return uint4{0, 0, 0, 0};
    };

    // Staged operands: this wave's 16 tokens x 128 columns, a lane taking
    // columns 4 (lane % 32) .. + 3 of tokens lane / 32 + 2 i.
    uint8_t *mine = lds + wave * (P * 16 * kPieceRow);
    const int sk = 4 * (lane & 31), sh = lane >> 5;
    float next[STAGE ? 8 : 1][4];
    auto fetch = [&](int mt, int slab) {
        if constexpr (STAGE) {
            const int k = slab * kMxSlab + sk;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = mt * 16 + sh + 2 * i;
                const T *p = x + (t < tokens ? t : 0) * j.ldx + k;
#pragma unroll
                for (int c = 0; c < 4; ++c) next[i][c] = 0.0f;
                if (t >= tokens || slab >= slabs) continue;
                if (vec && k + 4 <= j.K) {
                    if constexpr (TYPE == SGEMM_TYPE_F32) {
                        const f32v4 v = *(const f32v4 *)p;
#pragma unroll
                        for (int c = 0; c < 4; ++c) next[i][c] = v[c];
                    } else {
                        const uint2 v = *(const uint2 *)p;
                        const uint16_t h[4] = {(uint16_t)v.x, (uint16_t)(v.x >> 16), (uint16_t)v.y, (uint16_t)(v.y >> 16)};
#pragma unroll
                        for (int c = 0; c < 4; ++c) next[i][c] = MxType<TYPE>::load(&h[c]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (k + c < j.K) next[i][c] = MxType<TYPE>::load(p + c);
                }
            }
        }
    };
    auto stage = [&](int mt) {
        if constexpr (STAGE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (mt * 16 + 2 * i >= tokens) break;
                uint16_t p[4][P];
#pragma unroll
                for (int c = 0; c < 4; ++c) mx_split<P>(next[i][c], p[c]);
#pragma unroll
                for (int s = 0; s < P; ++s)
                    *(uint2 *)(mine + (s * 16 + sh + 2 * i) * kPieceRow + 2 * sk) =
                        uint2{(uint32_t)p[0][s] | (uint32_t)p[1][s] << 16, (uint32_t)p[2][s] | (uint32_t)p[3][s] << 16};
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    };

    f32v4 acc[R][MT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[r][mt] = f32v4{0.0f, 0.0f, 0.0f, 0.0f};

    if (STAGE) fetch(0, wave);
    for (int s0 = wave; s0 < slabs; s0 += kWaves * U) {
        MxBlock b[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
                b[u][r] = mx_block(row[r], words[r], plane, s0 + kWaves * u, q, s0 + kWaves * u < slabs);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int slab = s0 + kWaves * u;
            if (slab >= slabs) break;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (mt * 16 >= tokens) break;
                if constexpr (STAGE) {
                    stage(mt);
                    if (mt + 1 < MT && (mt + 1) * 16 < tokens) fetch(mt + 1, slab);
                    else fetch(0, slab + kWaves);
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint4 xs[P];
                    if constexpr (STAGE) {
                        const int t = mt * 16 + l16 < tokens ? l16 : tokens - 1 - mt * 16;   // unused columns: any token
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            xs[p] = *(const uint4 *)(mine + (p * 16 + t) * kPieceRow + 64 * q + 16 * s);
                    } else {
                        xs[0] = direct(mt, slab * kMxSlab + 32 * q + 8 * s);
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const uint32_t c = s == 0 ? b[u][r].codes.x : s == 1 ? b[u][r].codes.y
                                         : s == 2 ? b[u][r].codes.z : b[u][r].codes.w;
                        const bf16v8 w = mx_bf16x8(c, mx_scale(b[u][r], q));
#pragma unroll
                        for (int p = 0; p < P; ++p) acc[r][mt] = mx_mfma(w, xs[p], acc[r][mt]);
                    }
                }
                if constexpr (STAGE) {
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
            }
        }
    }

    // The waves' sums, added in wave order.  Lane l of a tile holds rows
    // 4 (l / 16) .. + 3 of W for token l % 16.
    __syncthreads();
    f32v4 *red = (f32v4 *)lds;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) red[((wave * R + r) * MT + mt) * 64 + lane] = acc[r][mt];
    __syncthreads();
    for (int i = tid; i < R * MT * 64; i += 64 * kWaves) {
        f32v4 sum = red[i];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += red[w * (R * MT * 64) + i];
        const int l = i & 63, mt = (i >> 6) % MT, r = (i >> 6) / MT;
        const int t = mt * 16 + (l & 15), n = n0 + 16 * r + 4 * (l >> 4);
        if (t >= tokens) continue;
        T *y = (T *)j.y + (m0 + t) * j.ldy + n;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (n + c < j.N) y[c] = MxType<TYPE>::from(sum[c]);
    }
}

template <int TYPE, bool STAGE, int R, int MT>
hipError_t launch_shape(const MxLinearJob &job, int vec, hipStream_t s) {
    MxLinearJob j = job;
    const int staged = STAGE ? kWaves * mx_pieces(TYPE) * 16 * kPieceRow : 0, sums = kWaves * R * MT * 1024;
    const int bytes = staged > sums ? staged : sums;
    const void *k = (const void *)linear_kernel<TYPE, STAGE, R, MT>;
    const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    void *params[] = {&j, &vec};
    const int64_t esize = TYPE == SGEMM_TYPE_F32 ? 4 : 2;
    constexpr int kMost = 65535 * 16 * MT;   // rows of one launch (the grid's y limit)
    for (int64_t m = 0; m < job.M; m += kMost) {
        j.M = job.M - m < kMost ? (int)(job.M - m) : kMost;
        j.x = (const char *)job.x + m * job.ldx * esize;
        j.y = (char *)job.y + m * job.ldy * esize;
        const hipError_t l = hipLaunchKernel(
            k, dim3((unsigned)((j.N + 16 * R - 1) / (16 * R)), (unsigned)((j.M + 16 * MT - 1) / (16 * MT))),
            dim3(64 * kWaves), params, bytes, s);
        if (l != hipSuccess) return l;
    }
    return hipSuccess;
}

template <int TYPE, bool STAGE>
hipError_t launch_tokens(const MxLinearJob &j, int vec, hipStream_t s) {
    if (j.M <= 16) return launch_shape<TYPE, STAGE, 1, 1>(j, vec, s);
    if (j.M <= 32) return launch_shape<TYPE, STAGE, 1, 2>(j, vec, s);
    return launch_shape<TYPE, STAGE, 2, 4>(j, vec, s);
}

}  // namespace

hipError_t launch_mx4_linear(const MxLinearJob &j, hipStream_t s) {
    // Rows on 16-byte boundaries (8 for the staged 16-bit loads would do).
    const int64_t bytes = j.type == SGEMM_TYPE_F32 ? 4 : 2;
    const int vec = ((uintptr_t)j.x & 15) == 0 && (j.ldx * bytes & 15) == 0;
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_tokens<SGEMM_TYPE_F32, true>(j, vec, s);
    case SGEMM_TYPE_F16: return launch_tokens<SGEMM_TYPE_F16, true>(j, vec, s);
    case SGEMM_TYPE_BF16:
        return vec ? launch_tokens<SGEMM_TYPE_BF16, false>(j, vec, s) : launch_tokens<SGEMM_TYPE_BF16, true>(j, vec, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace sgemm
