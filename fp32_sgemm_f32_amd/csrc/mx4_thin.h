// The products of a few float rows ("tokens") with 4-bit weights, shared by
// the thin product and the expert layer.
//
// A workgroup of 8 waves owns a piece of K and streams rows of weights past
// it; where K is short, sets of WK < 8 waves own it and share the rows.  A
// wave keeps its tokens' part of KS adjacent slabs (128 columns each) in
// operand registers for as long as it lives and takes 16 rows of weights and
// those slabs at a time, on v_mfma_f32_16x16x32_bf16 with the weights as the
// first operand: lane l holds the 16 bytes (one block, 32 codes) of row l % 16
// and block q = l / 16 of a slab, and step j = 0..3 takes codes 8 j .. 8 j + 7
// of every lane.  The sum's order along K does not matter as long as the
// tokens follow it, so they are taken at column 32 q + 8 j.  Two slabs are
// loaded as 8 rows x 128 bytes, whole lines of memory, and exchanged between
// lanes l and l ^ 8 (`up` of 128 experts x 4096 x 1536: 160 us, by 16 rows x
// 64 bytes 180).  The waves' sums meet in LDS and are added in wave order, G
// tiles of rows at a time.
//
// (A wave that took the tokens anew for every 16 rows read four to twelve
// bytes of them for each byte of weights and split them again each time: 13
// fp32 tokens x 16384 against 5001 rows took 71 us.)
//
// Nothing is rounded on the way in.  A code times its scale is exact in bf16
// (two bits of significand; the conversion instruction applies the scale).  A
// token value is cut into P bf16 pieces that add up to it: one for bf16, two
// for fp16 (11 bits), three for fp32 (24 bits); each piece costs one more
// matrix step and as many registers.  With at most 8 (two pieces) or 5 (three)
// tokens they are folded: the pieces take the other columns of the same step,
// and their sums are added with the waves'.  bf16 ends at 2^-133, so where all
// of a wave's values of an fp32 token lie below 2^-60 they are taken 2^32 times
// larger and the wave's sum 2^32 times smaller: both exact, and far from
// overflow with the largest weight.
//
// A code under a scale byte of 253 or 254 can exceed the largest float, though
// its products need not.  As bf16 it is infinite, and its product with a zero
// piece of a token NaN: it always shows in the sum.  So a wave that met an
// infinite sum or NaN looks its rows over at the end and computes those that
// hold such a weight anew, in plain floats from memory.
#pragma once

#include "mx4.h"

namespace sgemm {

constexpr int kThinWaves = 8, kThinThreads = 64 * kThinWaves;
constexpr int mx_pieces(int type) { return type == SGEMM_TYPE_BF16 ? 1 : type == SGEMM_TYPE_F16 ? 2 : 3; }

// Codes 0..7 of a register, times the scale, as bf16.
__device__ __forceinline__ bf16v8 mx_bf16x8(uint32_t codes, float scale) {
    const bf16v2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16v2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16v2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16v2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16v8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// v as P bf16 pieces, cut (not rounded) from the top.  An infinity or NaN
// stays whole in the first.
template <int P>
__device__ __forceinline__ void mx_split(float v, uint16_t (&p)[P]) {
    const uint32_t b = __float_as_uint(v);
    const bool finite = (b & 0x7f800000u) != 0x7f800000u;
    p[0] = (uint16_t)(b >> 16 | ((b & 0x7fffffffu) > 0x7f800000u ? 0x40u : 0u));
    float rest = finite ? v - __uint_as_float(b & 0xffff0000u) : 0.0f;
#pragma unroll
    for (int i = 1; i < P; ++i) {
        const uint32_t r = __float_as_uint(rest);
        p[i] = (uint16_t)(r >> 16);
        rest -= __uint_as_float(r & 0xffff0000u);
    }
}

// Eight values as P operand registers of 16 bytes.
template <int P>
__device__ __forceinline__ void mx_split8(const float (&v)[8], uint4 (&x)[P]) {
    uint16_t p[8][P];
#pragma unroll
    for (int i = 0; i < 8; ++i) mx_split<P>(v[i], p[i]);
#pragma unroll
    for (int k = 0; k < P; ++k)
        x[k] = uint4{(uint32_t)p[0][k] | (uint32_t)p[1][k] << 16, (uint32_t)p[2][k] | (uint32_t)p[3][k] << 16,
                     (uint32_t)p[4][k] | (uint32_t)p[5][k] << 16, (uint32_t)p[6][k] | (uint32_t)p[7][k] << 16};
}

// The same for P > 1 and finite values, in half the instructions: the first
// piece is cut (rounded, the largest floats would become infinite), the
// others are rounded to nearest, two at a time; of three the last is exact.
template <int P>
__device__ __forceinline__ void mx_split8_finite(const float (&v)[8], uint4 (&x)[P]) {
    uint32_t w[P][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
        w[0][i] = __builtin_amdgcn_perm(b, a, 0x07060302u);   // the upper halves of both
        float ra = v[2 * i] - __uint_as_float(a & 0xffff0000u), rb = v[2 * i + 1] - __uint_as_float(b & 0xffff0000u);
#pragma unroll
        for (int k = 1; k < P; ++k) {
            const bf16v2 p{(__bf16)ra, (__bf16)rb};
            w[k][i] = __builtin_bit_cast(uint32_t, p);
            ra -= __uint_as_float(w[k][i] << 16);
            rb -= __uint_as_float(w[k][i] & 0xffff0000u);
        }
    }
#pragma unroll
    for (int k = 0; k < P; ++k) x[k] = uint4{w[k][0], w[k][1], w[k][2], w[k][3]};
}

// Eight bf16 values of a row from column c on, zeros at and after `cols`.
__device__ __forceinline__ uint4 mx_bf16_edge8(const uint16_t *row, int c, int cols) {
    if (c + 8 <= cols) return __builtin_bit_cast(uint4, *(const u32v4_any *)(row + c));
    uint32_t u[4] = {0, 0, 0, 0};
    if (c < cols)
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) u[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
    return uint4{u[0], u[1], u[2], u[3]};
}

// What fp32 values whose largest magnitude has these bits are multiplied by.
__device__ __forceinline__ float mx_lift(uint32_t largest) { return largest < 0x21800000u ? 0x1p32f : 1.0f; }

// A wave's tokens: MT tiles, KS slabs, P pieces; WK waves share K.  FOLD: the
// pieces of a token stand in different columns.
template <int TYPE, int P, int KS, int WK, int MT, bool FOLD = false>
struct MxTokens {
    typedef typename MxType<TYPE>::T T;
    static constexpr int Q = FOLD ? 1 : P;              // matrix steps for a product
    static constexpr int kFold = FOLD ? P : 1, kTokens = 16 / kFold;   // columns of a token, tokens of a tile
    uint4 x[KS][MT][4][Q];
    float back[MT];   // what sums of a token are multiplied by

    // The token of the lane's column (-1: none) and the piece that stands there.
    static __device__ __forceinline__ int token() {
        const int c = threadIdx.x & 15;
        return c < kFold * kTokens ? c % kTokens : -1;
    }
    static __device__ __forceinline__ int piece() { return (threadIdx.x & 15) / kTokens; }
    // One operand of the pieces of eight values.
    static __device__ __forceinline__ void take(const uint4 (&all)[P], uint4 (&to)[Q]) {
        if constexpr (FOLD) {
            const int p = piece();
            to[0] = all[0];
#pragma unroll
            for (int k = 1; k < P; ++k)
                if (p == k) to[0] = all[k];
        } else {
#pragma unroll
            for (int k = 0; k < P; ++k) to[k] = all[k];
        }
    }

    // The lane's tokens are in row[mt] (NULL: none, zeros), its columns in
    // slabs slab0 + i.
    __device__ __forceinline__ void load(const T *const (&row)[MT], int slab0, int cols, int q) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            back[mt] = 1.0f;
            if constexpr (TYPE == SGEMM_TYPE_BF16 && P == 1) {
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int c = (slab0 + i) * kMxSlab + 32 * q + 8 * s;
                        x[i][mt][s][0] = row[mt] ? mx_bf16_edge8(row[mt], c, cols) : uint4{0, 0, 0, 0};
                    }
            } else if constexpr (TYPE != SGEMM_TYPE_F32) {
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        float v[8];
                        uint4 all[P];
                        mx_load_edge8<TYPE>(row[mt], (slab0 + i) * kMxSlab + 32 * q + 8 * s, row[mt] ? cols : 0, v);
                        mx_split8<P>(v, all);
                        take(all, x[i][mt][s]);
                    }
            } else {
                float v[KS][4][8];
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        mx_load_edge8<TYPE>(row[mt], (slab0 + i) * kMxSlab + 32 * q + 8 * s, row[mt] ? cols : 0, v[i][s]);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t b = __float_as_uint(v[i][s][k]) & 0x7fffffffu;
                            m = m > b ? m : b;
                        }
                    }
                // The token's other blocks lie with lanes l ^ 16, l ^ 32, l ^ 48.
                uint32_t o = __shfl_xor(m, 16, 64);
                m = m > o ? m : o;
                o = __shfl_xor(m, 32, 64);
                m = m > o ? m : o;
                const float lift = mx_lift(m);
                back[mt] = lift == 1.0f ? 1.0f : 0x1p-32f;
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        uint4 all[P];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[i][s][k] *= lift;
                        if (m < 0x7f800000u) mx_split8_finite<P>(v[i][s], all);
                        else mx_split8<P>(v[i][s], all);
                        take(all, x[i][mt][s]);
                    }
            }
        }
    }

    // The same from pieces in memory: piece p of a row at row + p * stride,
    // `cols` a multiple of 8, rows 16-byte aligned.
    __device__ __forceinline__ void load_pieces(const uint16_t *row, int64_t stride, int slab0, int cols, int q) {
        static_assert(MT == 1 && TYPE == SGEMM_TYPE_BF16, "one tile");
        back[0] = 1.0f;
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int p = 0; p < Q; ++p) {
                    const int c = (slab0 + i) * kMxSlab + 32 * q + 8 * s;
                    x[i][0][s][p] = row && c < cols ? *(const uint4 *)(row + (FOLD ? piece() : p) * stride + c) : uint4{0, 0, 0, 0};
                }
    }
};

// Sums in LDS of a stream.
template <int G, int MT>
constexpr int kThinSums = 2 * kThinWaves * G * MT * 64;

// A lane's weights of one slab: its block's codes and scale.
struct MxBlock {
    uint4 codes;
    uint32_t word;   // the slab's four scale bytes of the row
};

__device__ __forceinline__ float mx_scale(const MxBlock &b, int q) {
    return __uint_as_float((b.word >> (8 * q) & 255u) << 23);
}

__device__ __forceinline__ f32v4 mx_mfma(bf16v8 w, uint4 x, f32v4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16v8, x), acc, 0, 0, 0);
}

// A 4-bit matrix as the kernels take it.
struct MxWeights {
    const uint8_t *codes;
    const uint32_t *words;
    int64_t rowb, plane;   // bytes of a row of codes, words of a plane of scales
    int slabs;

    // Zeros past the last slab.
    template <bool NT>
    __device__ __forceinline__ uint4 codes16(int64_t row, int slab, int q) const {
        if (slab >= slabs) return uint4{0, 0, 0, 0};
        const i32v4 *p = (const i32v4 *)(codes + row * rowb + (int64_t)slab * kMxSlabBytes + 16 * q);
        return __builtin_bit_cast(uint4, NT ? __builtin_nontemporal_load(p) : *p);
    }
    __device__ __forceinline__ uint32_t word(int64_t row, int slab) const { return slab < slabs ? words[slab * plane + row] : 0; }
    __device__ __forceinline__ MxBlock load(int64_t row, int slab, int q) const {
        return MxBlock{codes16<true>(row, slab, q), word(row, slab)};
    }
};

__device__ __forceinline__ bool mx_finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// The four floats of v whose bits are set in `rows`.
__device__ __forceinline__ void mx_store_rows(float *p, f32v4 v, int rows) {
    if (rows == 15) {
        *(f32v4 *)p = v;
        return;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (rows >> c & 1) p[c] = v[c];
}

// Whether row r holds a weight beyond the largest float in slabs [from, to):
// from 2 on under scale byte 254, from 4 on under 253.  For a whole wave.
__device__ __forceinline__ bool mx_beyond(const MxWeights &w, int64_t r, int from, int to) {
    const int lane = threadIdx.x & 63;
    uint32_t hit = 0;
#pragma nounroll
    for (int b0 = 4 * from; b0 < 4 * to; b0 += 64) {
        const int block = b0 + lane;
        const uint32_t s = block < 4 * to ? w.word(r, block >> 2) >> (8 * (block & 3)) & 255u : 0;
        if (s - 253u < 2u) {
            const uint4 c = *(const uint4 *)(w.codes + r * w.rowb + (int64_t)block * 16);
            hit |= s == 254 ? (c.x | c.y | c.z | c.w) & 0x44444444u
                            : ((c.x & c.x >> 1) | (c.y & c.y >> 1) | (c.z & c.z >> 1) | (c.w & c.w >> 1)) & 0x22222222u;
        }
    }
    return __any(hit != 0);
}

// The sum over slabs [from, to) of row r times a token, whose value at a column
// (zero beyond the last one) is value(column).  In plain floats, of a quarter of
// the weights: those are exact from 2^-130 to 1.5 2^127.  For a whole wave.
template <class Value>
__device__ __forceinline__ float mx_plain_sum(const MxWeights &w, int64_t r, int from, int to, Value value) {
    const int lane = threadIdx.x & 63;
    float quarter = 0.0f;
#pragma nounroll
    for (int b0 = 4 * from; b0 < 4 * to; b0 += 64) {
        const int block = b0 + lane;
        if (block >= 4 * to) break;
        const uint32_t s = w.word(r, block >> 2) >> (8 * (block & 3)) & 255u;
        const float f = s == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(1.0f, (int)s - 129);
#pragma nounroll
        for (int k = 0; k < 16; ++k) {
            const auto two = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.codes[r * w.rowb + (int64_t)block * 16 + k], 1.0f, 0);
            quarter = fmaf(value(block * 32 + 2 * k), two[0] * f, quarter);
            quarter = fmaf(value(block * 32 + 2 * k + 1), two[1] * f, quarter);
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) quarter += __shfl_xor(quarter, off, 64);
    return 4.0f * quarter;
}

inline __host__ __device__ MxWeights mx_weights(const uint8_t *codes, const uint8_t *scales, int64_t rows, int cols) {
    return MxWeights{codes, (const uint32_t *)scales, (int64_t)mx_slabs(cols) * kMxSlabBytes, mx_plane_rows(rows), mx_slabs(cols)};
}

// Streams row tiles [first, end) past the tokens.  WK waves share K,
// kThinWaves / WK sets of them the row tiles; a wave takes G tiles at a time,
// U of them next to each other (whose sums one thread then holds), and loads
// the next G while it multiplies.
// NT: the weights are read past the caches (used once, and more of them than
// the caches hold).
template <int U, int G, int KS, int WK, bool NT>
struct MxStream {
    static_assert(G % U == 0, "whole units in a group");
    static constexpr int WR = kThinWaves / WK;
    MxBlock b[G][KS];

    // Slot g's tile in the group that begins at t0.
    static __device__ __forceinline__ int tile_of(int t0, int g) {
        return t0 + g / U * (WR * U) + (int)(threadIdx.x >> 6) / WK * U + g % U;
    }
    // Whether slabs i and i + 1 are loaded together.
    static constexpr bool pair(int i) { return i % 2 == 0 && i + 1 < KS; }

    // Sends for slab i, or the pair i, i + 1, of every slot's tile in the group
    // that begins at t0 (past the end: nothing; what is computed from what
    // the registers hold is dropped).
    template <class Row>
    __device__ __forceinline__ void fetch(const MxWeights &w, int slab0, int i, int t0, int end, Row row) {
        const int m = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int tile = tile_of(t0, g);
            if (tile >= end) continue;
            const int64_t r = row(tile, m);
            if (pair(i)) {
                b[g][i].codes = w.codes16<NT>(row(tile, m & 7), slab0 + i + (m >> 3), q);
                b[g][i + 1].codes = w.codes16<NT>(row(tile, 8 + (m & 7)), slab0 + i + (m >> 3), q);
                b[g][i + 1].word = w.word(r, slab0 + i + 1);
            } else {
                b[g][i].codes = w.codes16<NT>(r, slab0 + i, q);
            }
            b[g][i].word = w.word(r, slab0 + i);
        }
    }

    // The registers of a pair as loaded -> slab i and slab i + 1 of row l % 16.
    __device__ __forceinline__ void exchange(uint4 &x, uint4 &y) {
        const bool upper = threadIdx.x & 8;
        const auto one = [&](uint32_t &p, uint32_t &r) {
            const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)(upper ? p : r), 0x128, 15, 15, true);   // of lane l ^ 8
            if (upper) p = got;
            else r = got;
        };
        one(x.x, y.x), one(x.y, y.y), one(x.z, y.z), one(x.w, y.w);
    }

    // Sends for the first group's weights; row(tile, m) is row m of a tile,
    // slab0 the wave's first slab.
    template <class Row>
    __device__ __forceinline__ void begin(const MxWeights &w, int slab0, int first, int end, Row row) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < KS; ++i) b[g][i] = MxBlock{uint4{0, 0, 0, 0}, 0};
#pragma unroll
        for (int i = 0; i < KS; i += pair(i) ? 2 : 1) fetch(w, slab0, i, first, end, row);
    }

    // After begin with the same arguments.  emit(tile, mt, l, sums, rows) takes
    // the sums of U tiles (tile .. tile + U - 1) for token l % 16 of tile mt, rows
    // 4 (l / 16) + c of each where bit c of `rows` is set.  red: LDS for kThinSums<G, MT> sums.
    // odd is set, for the whole wave, where a sum of the last piece is infinite
    // or NaN.
    // With K in several pieces, carry (LDS, (end - first) * MT * 64 sums)
    // holds them from the first piece to the last.  Every thread of the
    // workgroup calls this.
    template <int TYPE, int P, int MT, bool FOLD, class Row, class Emit>
    __device__ __forceinline__ void run(const MxTokens<TYPE, P, KS, WK, MT, FOLD> &x, const MxWeights &w, int slab0, int first, int end,
                                        f32v4 *red, f32v4 *carry, bool first_piece, bool last_piece, bool &odd, Row row, Emit emit) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane >> 4;
        for (int t0 = first; t0 < end; t0 += G * WR) {
            f32v4 acc[G][MT];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[g][mt] = f32v4{0.0f, 0.0f, 0.0f, 0.0f};
            // The G tiles in turn: their products do not wait for each other.
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                if (pair(i)) {
#pragma unroll
                    for (int g = 0; g < G; ++g) exchange(b[g][i].codes, b[g][i + 1 < KS ? i + 1 : i].codes);
                }
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const uint4 c = b[g][i].codes;
                        const bf16v8 v = mx_bf16x8(s == 0 ? c.x : s == 1 ? c.y : s == 2 ? c.z : c.w, mx_scale(b[g][i], q));
#pragma unroll
                        for (int p = 0; p < (FOLD ? 1 : P); ++p)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) acc[g][mt] = mx_mfma(v, x.x[i][mt][s][p], acc[g][mt]);
                    }
                if (!pair(i)) fetch(w, slab0, i % 2 == 1 ? i - 1 : i, t0 + G * WR, end, row);
            }
            // Two halves of red in turn: one meeting for a group.
            f32v4 *half = red + ((t0 - first) / (G * WR) & 1) * (kThinWaves * G * MT * 64);
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if constexpr (TYPE == SGEMM_TYPE_F32) acc[g][mt] *= x.back[mt];
                    half[((wave * G + g) * MT + mt) * 64 + lane] = acc[g][mt];
                }
            __syncthreads();
            bool here = false;
            for (int i = tid; i < G / U * WR * MT * 64; i += kThinThreads) {
                const int l = i & 63, mt = (i >> 6) % MT, unit = (i >> 6) / MT, set = unit % WR, g = unit / WR * U;
                if (t0 + unit * U >= end) break;
                if (FOLD && (l & 15) >= x.kTokens) continue;
                f32v4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const f32v4 *from = half + ((set * WK * G + g + u) * MT + mt) * 64 + l;
                    v[u] = *from;
#pragma unroll
                    for (int k = 1; k < WK; ++k) v[u] += from[k * G * MT * 64];
                    if constexpr (FOLD) {
#pragma unroll
                        for (int f = 1; f < P; ++f)
#pragma unroll
                            for (int k = 0; k < WK; ++k) v[u] += from[k * G * MT * 64 + f * x.kTokens];
                    }
                    f32v4 *kept = carry + ((t0 - first + unit * U + u) * MT + mt) * 64 + l;
                    if (!first_piece) v[u] = *kept + v[u];
                    if (!last_piece) *kept = v[u];
                }
                if (last_piece) {
                    f32v4 all = v[0];
#pragma unroll
                    for (int u = 1; u < U; ++u) all += v[u];
                    here |= !mx_finite(all[0] + all[1] + (all[2] + all[3]));
                    emit(t0 + unit * U, mt, l, v, 15);
                }
            }
            odd |= __builtin_amdgcn_readfirstlane(__any(here)) != 0;
        }
        __syncthreads();   // red is free
    }

    // Gives emit this wave's sums of slabs [from, to) once more for the rows that
    // hold a weight beyond the largest float; value(mt, t, column): token t of
    // tile mt, zero beyond the last column.
    template <int MT, int TOKENS, class Row, class Value, class Emit>
    static __device__ __forceinline__ void mend(const MxWeights &w, int from, int to, int first, int end, Row row, Value value, Emit emit) {
        if (to > w.slabs) to = w.slabs;
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma nounroll
        for (int t0 = first; t0 < end; t0 += G * WR)
#pragma nounroll
            for (int i = wave; i < G / U * WR * MT; i += kThinWaves) {
                const int mt = i % MT, tile = t0 + i / MT * U;
                if (tile >= end) break;
#pragma nounroll
                for (int m = 0; m < 16; ++m) {
                    bool beyond = false;
#pragma nounroll
                    for (int u = 0; u < U; ++u) beyond |= mx_beyond(w, row(tile + u, m), from, to);
                    if (!beyond) continue;
#pragma nounroll
                    for (int t = 0; t < TOKENS; ++t) {
                        f32v4 v[U];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const float sum = mx_plain_sum(w, row(tile + u, m), from, to, [&](int column) { return value(mt, t, column); });
                            v[u] = f32v4{sum, sum, sum, sum};
                        }
                        if (lane == (m >> 2) * 16 + t) emit(tile, mt, lane, v, 1 << (m & 3));
                    }
                }
            }
    }
};

// The kernel's arguments (one struct), read again: what rare code at a kernel's
// end needs of them is kept in no register until then.
template <class A>
__device__ __forceinline__ A mx_arguments() {
    typedef const __attribute__((address_space(4))) A Argument;
    uint64_t p = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    A a;
    __builtin_memcpy(&a, (const void *)(Argument *)p, sizeof(A));
    return a;
}

// The number of row tiles each workgroup of `groups` takes.
inline int mx_share(int tiles, int groups, int unit) {
    const int per = (tiles + groups - 1) / groups;
    return (per + unit - 1) / unit * unit;
}

struct MxLinearJob {
    const void *x;
    int64_t ldx;
    const uint8_t *codes, *scales;
    int M, N, K, type;
    void *y;
    int64_t ldy;
    float *scratch;
};

struct MxMoeJob {
    const void *x, *router;
    int64_t ldx, ldr;
    const uint8_t *up, *sup, *down, *sdown;
    int tokens, hidden, inner, experts, top, norm, type;
    void *y;
    int64_t ldy;
    char *scratch;
};

hipError_t launch_mx4_linear(const MxLinearJob &j, hipStream_t s);
int64_t mx4_linear_scratch(int M, int N, int K, int type);
hipError_t launch_mx4_moe(const MxMoeJob &j, hipStream_t s);
int64_t mx4_moe_scratch(int tokens, int hidden, int inner, int experts, int top);

}  // namespace sgemm
