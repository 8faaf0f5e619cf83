// The gated activation H = silu(G) * U of GU = [G, U], with an 8-bit checkpoint
// of G and U in groups of 128 columns, and its gradient from that checkpoint:
//
//     p = 1 / (1 + exp(-g))     h = g p u
//     dg = dh u p (1 + g (1 - p))     du = dh g p
//
// with the checkpoint's g and u in the gradient.  In fp32 (far gates in 64 bits),
// rounded once.
//
// Bound by HBM: a lane takes eight columns of G and the same of U, so that
// every value is read and written once (8192 x 14336 bf16: 0.95 GB each way in 192
// us, 4.9 TB/s, and 194).
#include "i8.h"

namespace sgemm {
namespace {

// Below this exp(g) leaves the normal numbers of fp32 and exp(-g) its range,
// while exp(g) times what it meets (u or dh up to 1e38) need not be small: such
// gates, 1 + exp(g) = 1, are taken in 64 bits from the square of exp(g / 2).
// What a lane knows of its gates' magnitudes says whether to look for them, which
// it does behind its stores, writing again: hardly any does, and before the stores
// the others take 3% longer (8192 x 14336 and 4096 x 4096 bf16; so no longer than
// without).
constexpr float kFarGate = -87.0f;
__device__ __forceinline__ double i8_far_gate(float g) {
    const double e = expf(0.5f * g);
    return e * e;
}

template <int TYPE>
__global__ __launch_bounds__(256) void i8_swiglu_forward_kernel(I8SwigluJob j) {
    typedef typename MxType<TYPE>::T E;
    const int chunks = (int)(i8_ld(j.inner) / 8);
    const I8Place at = i8_place(chunks, 256);
    const bool real = at.row < j.rows;
    const E *x = (const E *)j.x + (real ? at.row : 0) * j.ldx;
    float g[8], u[8], h[8];
    mx_load_edge8<TYPE>(x, at.c, real ? j.inner : 0, g);
    mx_load_edge8<TYPE>(x + j.inner, at.c, real ? j.inner : 0, u);
    const uint32_t most = i8_max8(g);
    const float sg = i8_scale(i8_max16(most), kI8Levels), su = i8_scale(i8_max16(i8_max8(u)), kI8Levels);
    if (!real) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = g[i] / (1.0f + expf(-g[i])) * u[i];
    const int64_t q = at.row * chunks * 8 + at.c;
    *(uint2 *)(j.gq + q) = i8_nearest8(g, sg, 1.0f / sg);
    *(uint2 *)(j.uq + q) = i8_nearest8(u, su, 1.0f / su);
    if ((threadIdx.x & 15) == 0) j.gs[q / 128] = sg, j.us[q / 128] = su;
    i8_store8<TYPE>((E *)j.y + at.row * j.ldy, at.c, j.inner, h);
    if (__builtin_expect(most > i8_magnitude(kFarGate), 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (g[i] < kFarGate) h[i] = (float)((double)g[i] * u[i] * i8_far_gate(g[i]));
        i8_store8<TYPE>((E *)j.y + at.row * j.ldy, at.c, j.inner, h);
    }
}

template <int TYPE>
__global__ __launch_bounds__(256) void i8_swiglu_backward_kernel(I8SwigluJob j) {
    typedef typename MxType<TYPE>::T E;
    const int chunks = (j.inner + 7) / 8;
    const I8Place at = i8_place(chunks, 256);
    if (at.row >= j.rows) return;
    const int64_t q = at.row * i8_ld(j.inner) + at.c;
    float g[8], u[8], d[8], dg[8], du[8];
    mx_load_edge8<TYPE>((const E *)j.x + at.row * j.ldx, at.c, j.inner, d);
    const float sg = j.gs[q / 128];
    i8_values8(*(const uint2 *)(j.gq + q), sg, g);
    i8_values8(*(const uint2 *)(j.uq + q), j.us[q / 128], u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // 1 - p as it is: for large g it is exp(-g) p, of which the difference would lose the last bits.
        const float e = expf(-g[i]), p = 1.0f / (1.0f + e), rest = g[i] > 0.0f ? e * p : 1.0f - p;
        dg[i] = d[i] * u[i] * p * (1.0f + g[i] * rest);
        du[i] = d[i] * (g[i] * p);
    }
    E *y = (E *)j.y + at.row * j.ldy;
    i8_store8<TYPE>(y, at.c, j.inner, dg);
    i8_store8<TYPE>(y + j.inner, at.c, j.inner, du);
    if (__builtin_expect(fabsf(kI8Levels * sg) > -kFarGate, 0)) {
        // One value at a time, read again: nothing is kept in registers for this.
        const E *x = (const E *)j.x + at.row * j.ldx;
        for (int i = 0; i < 8 && at.c + i < j.inner; ++i) {
            const float gate = (float)j.gq[q + i] * sg;
            if (!(gate < kFarGate)) continue;
            const double dp = MxType<TYPE>::load(x + at.c + i) * i8_far_gate(gate), up = (float)j.uq[q + i] * j.us[q / 128];
            y[at.c + i] = MxType<TYPE>::from((float)(dp * up * (1.0 + gate)));
            y[j.inner + at.c + i] = MxType<TYPE>::from((float)(dp * gate));
        }
    }
}

const void *forward_kernel(int type) {
    switch (type) {
    case SGEMM_TYPE_F32: return (const void *)i8_swiglu_forward_kernel<SGEMM_TYPE_F32>;
    case SGEMM_TYPE_BF16: return (const void *)i8_swiglu_forward_kernel<SGEMM_TYPE_BF16>;
    default: return (const void *)i8_swiglu_forward_kernel<SGEMM_TYPE_F16>;
    }
}
const void *backward_kernel(int type) {
    switch (type) {
    case SGEMM_TYPE_F32: return (const void *)i8_swiglu_backward_kernel<SGEMM_TYPE_F32>;
    case SGEMM_TYPE_BF16: return (const void *)i8_swiglu_backward_kernel<SGEMM_TYPE_BF16>;
    default: return (const void *)i8_swiglu_backward_kernel<SGEMM_TYPE_F16>;
    }
}

}  // namespace

hipError_t launch_i8_swiglu_forward(const I8SwigluJob &job, hipStream_t s) {
    I8SwigluJob j = job;
    void *params[] = {&j};
    return hipLaunchKernel(forward_kernel(j.type), dim3(i8_grid(j.rows, i8_ld(j.inner) / 8, 256)), dim3(256), params, 0, s);
}

hipError_t launch_i8_swiglu_backward(const I8SwigluJob &job, hipStream_t s) {
    I8SwigluJob j = job;
    void *params[] = {&j};
    return hipLaunchKernel(backward_kernel(j.type), dim3(i8_grid(j.rows, (j.inner + 7) / 8, 256)), dim3(256), params, 0, s);
}

}  // namespace sgemm
