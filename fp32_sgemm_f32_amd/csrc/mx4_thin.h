// The inner step of the products of a few float rows ("tokens") with 4-bit
// weights, shared by the thin product and the expert layer.
//
// A wave takes 16 rows of weights and one slab (128 columns) at a time and
// multiplies it with up to 16 tokens on v_mfma_f32_16x16x32_bf16, the weights
// as the first operand: lane l loads the 16 bytes (one block, 32 codes) of
// row l % 16 and block q = l / 16, so a wave reads 64 bytes of each row, and
// matrix step j = 0..3 takes codes 8 j .. 8 j + 7 of every lane.  The sum's
// order along K does not matter as long as the tokens follow it: they are
// taken at column 32 q + 8 j.
//
// Nothing is rounded on the way in.  A code times its scale is exact in bf16
// (two bits of significand; the conversion instruction applies the scale).
// A token value is given as P bf16 pieces that add up to it exactly: one for
// bf16, two for fp16 (11 bits), three for fp32 (24 bits); each piece costs
// one more matrix step, which the load of the weights hides.
#pragma once

#include "mx4.h"

namespace sgemm {

constexpr int mx_pieces(int type) { return type == SGEMM_TYPE_BF16 ? 1 : type == SGEMM_TYPE_F16 ? 2 : 3; }

// Codes 0..7 of a register, times the scale, as bf16.
__device__ __forceinline__ bf16v8 mx_bf16x8(uint32_t codes, float scale) {
    const bf16v2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16v2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16v2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16v2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16v8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// v as P bf16 pieces, cut (not rounded) from the top so that their sum is v.
// An infinity or NaN stays whole in the first.
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

// A lane's weights of one slab: its block's codes and scale.
struct MxBlock {
    uint4 codes;
    uint32_t word;   // the slab's four scale bytes of the row
};

__device__ __forceinline__ MxBlock mx_block(const uint8_t *row, const uint32_t *words, int64_t plane, int slab, int q,
                                            bool real) {
    MxBlock b{uint4{0, 0, 0, 0}, 0};
    if (real) {
        b.codes = *(const uint4 *)(row + (int64_t)slab * kMxSlabBytes + 16 * q);
        b.word = words[slab * plane];
    }
    return b;
}

__device__ __forceinline__ float mx_scale(const MxBlock &b, int q) {
    return __uint_as_float((b.word >> (8 * q) & 255u) << 23);
}

__device__ __forceinline__ f32v4 mx_mfma(bf16v8 w, uint4 x, f32v4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16v8, x), acc, 0, 0, 0);
}

struct MxLinearJob {
    const void *x;
    int64_t ldx;
    const uint8_t *codes, *scales;
    int M, N, K, type;
    void *y;
    int64_t ldy;
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
hipError_t launch_mx4_moe(const MxMoeJob &j, hipStream_t s);
int64_t mx4_moe_scratch(int tokens, int hidden, int inner, int experts, int top, int type);

}  // namespace sgemm
