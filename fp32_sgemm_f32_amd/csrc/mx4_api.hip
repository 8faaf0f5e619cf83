// C entry points of the 4-bit operators (declared in include/sgemm_f32.h):
// argument checks, then one launcher each.
#include <hip/hip_runtime_api.h>

#include "checks.h"
#include "mx4_thin.h"

namespace sgemm {
namespace {

bool dim_ok(int n) { return n >= 0 && n <= SGEMM_MX4_MAX_DIM; }
int64_t codes_bytes(int rows, int cols) { return (int64_t)rows * mx_slabs(cols) * kMxSlabBytes; }
int64_t scales_bytes(int rows, int cols) { return mx_plane_rows(rows) * 4 * mx_slabs(cols); }

Span codes(const void *p, int rows, int cols, bool out) { return Span{p, codes_bytes(rows, cols), 16, out}; }
Span scales(const void *p, int rows, int cols, bool out) { return Span{p, scales_bytes(rows, cols), 4, out}; }

}  // namespace
}  // namespace sgemm

using namespace sgemm;

SGEMM_API int sgemm_f32_mx4_bytes(int rows, int cols, long long *codes_out, long long *scales_out) {
    if (!dim_ok(rows) || !dim_ok(cols)) return SGEMM_ERR_SHAPE;
    if (codes_out) *codes_out = codes_bytes(rows, cols);
    if (scales_out) *scales_out = scales_bytes(rows, cols);
    return SGEMM_OK;
}

SGEMM_API int sgemm_f32_mx4_quantize(int rows, int cols, int type, const void *X, int ldx, int rule, void *c, void *s,
                                     void *ct, void *st, hipStream_t stream) {
    if (!dim_ok(rows) || !dim_ok(cols)) return SGEMM_ERR_SHAPE;
    if (!known_type(type) || (rule != SGEMM_MX4_SCALE_FLOOR && rule != SGEMM_MX4_SCALE_NOCLIP)) return SGEMM_ERR_CONFIG;
    if (rows == 0 || cols == 0) return SGEMM_OK;
    if (ldx < cols) return SGEMM_ERR_LD;
    const bool along = c || s, down = ct || st;
    if (!along && !down) return SGEMM_ERR_NULL;
    const Span spans[] = {floats(X, rows, cols, ldx, type, false),
                          codes(c, along ? rows : 0, cols, true), scales(s, along ? rows : 0, cols, true),
                          codes(ct, down ? cols : 0, rows, true), scales(st, down ? cols : 0, rows, true)};
    int dev = 0;
    const int status = check_spans(spans, &dev);
    if (status != SGEMM_OK) return status;
    return done(launch_mx4_quantize({X, ldx, rows, cols, type, rule == SGEMM_MX4_SCALE_NOCLIP, (uint8_t *)c, (uint8_t *)s,
                                     (uint8_t *)ct, (uint8_t *)st}, stream));
}

SGEMM_API int sgemm_f32_mx4_dequantize(int rows, int cols, const void *c, const void *s, int type, void *Y, int ldy,
                                       hipStream_t stream) {
    if (!dim_ok(rows) || !dim_ok(cols)) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (rows == 0 || cols == 0) return SGEMM_OK;
    if (ldy < cols) return SGEMM_ERR_LD;
    const Span spans[] = {codes(c, rows, cols, false), scales(s, rows, cols, false),
                          floats(Y, rows, cols, ldy, type, true)};
    int dev = 0;
    const int status = check_spans(spans, &dev);
    if (status != SGEMM_OK) return status;
    return done(launch_mx4_dequantize({(const uint8_t *)c, (const uint8_t *)s, rows, cols, type, Y, ldy}, stream));
}

SGEMM_API int sgemm_f32_mx4_gemm(int M, int N, int K, float alpha, const void *a, const void *sa, const void *b,
                                 const void *sb, float beta, int type, void *C, int ldc, hipStream_t stream) {
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (ldc < N) return SGEMM_ERR_LD;
    const int k = alpha == 0.0f ? 0 : K;   // nothing of A and B is read then
    if (K == 0) alpha = 0.0f;              // an empty sum stays zero whatever alpha
    const Span spans[] = {codes(a, M, k, false), scales(sa, M, k, false), codes(b, N, k, false),
                          scales(sb, N, k, false), floats(C, M, N, ldc, type, true)};
    int dev = 0, cus = 0;
    int status = check_spans(spans, &dev);
    if (status == SGEMM_OK) status = compute_units(dev, &cus);
    if (status != SGEMM_OK) return status;
    return done(launch_mx4_gemm({(const uint8_t *)a, (const uint8_t *)sa, (const uint8_t *)b, (const uint8_t *)sb, M, N, k,
                                 type, alpha, beta, C, ldc}, cus, stream));
}

// Scratch memory of a training step: the matrices that only one call needs,
// codes and scales 256-byte aligned.
namespace {

struct Packed {
    uint8_t *codes, *scales;
};

int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }
int64_t packed_bytes(int rows, int cols) { return up256(codes_bytes(rows, cols)) + up256(scales_bytes(rows, cols)); }
Packed packed_at(void *base, int64_t at, int rows, int cols) {
    uint8_t *p = (uint8_t *)base + at;
    return {p, p + up256(codes_bytes(rows, cols))};
}

// A matrix both ways; with rows == 0 or cols == 0 there is nothing to do.
MxQuantJob both_ways(const void *x, int ldx, int rows, int cols, int type, int rule, Packed q, Packed qt) {
    return {x, ldx, rows, cols, type, rule == SGEMM_MX4_SCALE_NOCLIP, q.codes, q.scales, qt.codes, qt.scales};
}

}  // namespace

SGEMM_API int sgemm_f32_mx4_train_scratch(int M, int N, int K, long long *forward, long long *backward) {
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return SGEMM_ERR_SHAPE;
    if (forward) *forward = packed_bytes(M, K) + packed_bytes(N, K);
    if (backward) *backward = packed_bytes(M, N) + packed_bytes(N, M);
    return SGEMM_OK;
}

SGEMM_API int sgemm_f32_mx4_train_forward(int M, int N, int K, int type, const void *X, int ldx, int type_w, const void *W,
                                          int ldw, int rule, void *Y, int ldy, void *xt, void *sxt, void *wt, void *swt,
                                          void *scratch, long long scratch_bytes, hipStream_t stream) {
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return SGEMM_ERR_SHAPE;
    if (!known_type(type) || !known_type(type_w) || (rule != SGEMM_MX4_SCALE_FLOOR && rule != SGEMM_MX4_SCALE_NOCLIP))
        return SGEMM_ERR_CONFIG;
    const bool x = M > 0 && K > 0, w = N > 0 && K > 0, y = M > 0 && N > 0;
    if ((x && ldx < K) || (w && ldw < K) || (y && ldy < N)) return SGEMM_ERR_LD;
    const int64_t need = packed_bytes(M, K) + packed_bytes(N, K);
    if (scratch && scratch_bytes < need) return SGEMM_ERR_SCRATCH;
    const Span spans[] = {floats(X, M, K, ldx, type, false), floats(W, N, K, ldw, type_w, false),
                          floats(Y, M, N, ldy, type, true), codes(xt, K, M, true), scales(sxt, K, M, true),
                          codes(wt, K, N, true), scales(swt, K, N, true), Span{scratch, need, 256, true}};
    int dev = 0, cus = 0;
    int status = check_spans(spans, &dev);
    if (status == SGEMM_OK) status = compute_units(dev, &cus);
    if (status != SGEMM_OK) return status;
    const Packed q = packed_at(scratch, 0, M, K), v = packed_at(scratch, packed_bytes(M, K), N, K);
    const MxQuantJob jx = both_ways(X, ldx, M, K, type, rule, q, {(uint8_t *)xt, (uint8_t *)sxt});
    const MxQuantJob jw = both_ways(W, ldw, N, K, type_w, rule, v, {(uint8_t *)wt, (uint8_t *)swt});
    hipError_t e = x && w ? launch_mx4_quantize_two(jx, jw, stream)
                   : x    ? launch_mx4_quantize(jx, stream)
                   : w    ? launch_mx4_quantize(jw, stream)
                          : hipSuccess;
    if (e == hipSuccess && y)
        e = launch_mx4_gemm({q.codes, q.scales, v.codes, v.scales, M, N, K, type, K > 0 ? 1.0f : 0.0f, 0.0f, Y, ldy}, cus, stream);
    return done(e);
}

SGEMM_API int sgemm_f32_mx4_train_backward(int M, int N, int K, int type, const void *dY, int ldd, int rule, const void *xt,
                                           const void *sxt, const void *wt, const void *swt, void *dX, int lddx, float beta,
                                           void *dW, int lddw, void *scratch, long long scratch_bytes, hipStream_t stream) {
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return SGEMM_ERR_SHAPE;
    if (!known_type(type) || (rule != SGEMM_MX4_SCALE_FLOOR && rule != SGEMM_MX4_SCALE_NOCLIP)) return SGEMM_ERR_CONFIG;
    const bool d = M > 0 && N > 0, x = M > 0 && K > 0, w = N > 0 && K > 0;
    if ((d && ldd < N) || (x && lddx < K) || (w && lddw < K)) return SGEMM_ERR_LD;
    const int64_t need = packed_bytes(M, N) + packed_bytes(N, M);
    if (scratch && scratch_bytes < need) return SGEMM_ERR_SCRATCH;
    const Span spans[] = {floats(dY, M, N, ldd, type, false), codes(xt, K, M, false), scales(sxt, K, M, false),
                          codes(wt, K, N, false), scales(swt, K, N, false), floats(dX, M, K, lddx, type, true),
                          floats(dW, N, K, lddw, SGEMM_TYPE_F32, true), Span{scratch, need, 256, true}};
    int dev = 0, cus = 0;
    int status = check_spans(spans, &dev);
    if (status == SGEMM_OK) status = compute_units(dev, &cus);
    if (status != SGEMM_OK) return status;
    const Packed q = packed_at(scratch, 0, M, N), qt = packed_at(scratch, packed_bytes(M, N), N, M);
    hipError_t e = d ? launch_mx4_quantize(both_ways(dY, ldd, M, N, type, rule, q, qt), stream) : hipSuccess;
    const MxGemmJob gx{q.codes, q.scales, (const uint8_t *)wt, (const uint8_t *)swt, M, K, N, type, N > 0 ? 1.0f : 0.0f, 0.0f, dX,
                       lddx};
    const MxGemmJob gw{qt.codes, qt.scales, (const uint8_t *)xt, (const uint8_t *)sxt, N, K, M, SGEMM_TYPE_F32,
                       M > 0 ? 1.0f : 0.0f, beta, dW, lddw};
    if (e == hipSuccess) e = x && w ? launch_mx4_gemm_two(gx, gw, cus, stream)
                             : x    ? launch_mx4_gemm(gx, cus, stream)
                             : w    ? launch_mx4_gemm(gw, cus, stream)
                                    : hipSuccess;
    return done(e);
}

SGEMM_API int sgemm_f32_mx4_linear_scratch(int M, int N, int K, int type, long long *bytes) {
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (!bytes) return SGEMM_ERR_NULL;
    *bytes = mx4_linear_scratch(M, N, K, type);
    return SGEMM_OK;
}

SGEMM_API int sgemm_f32_mx4_linear(int M, int N, int K, int type, const void *X, int ldx, const void *c, const void *s,
                                   void *Y, int ldy, void *scratch, long long scratch_bytes, hipStream_t stream) {
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (ldx < K || ldy < N) return SGEMM_ERR_LD;
    const int64_t need = mx4_linear_scratch(M, N, K, type);
    if (scratch && scratch_bytes < need) return SGEMM_ERR_SCRATCH;
    const Span spans[] = {floats(X, M, K, ldx, type, false), codes(c, N, K, false), scales(s, N, K, false),
                          floats(Y, M, N, ldy, type, true), Span{scratch, need, 256, true}};
    int dev = 0;
    const int status = check_spans(spans, &dev);
    if (status != SGEMM_OK) return status;
    return done(launch_mx4_linear({X, ldx, (const uint8_t *)c, (const uint8_t *)s, M, N, K, type, Y, ldy, (float *)scratch},
                                  stream));
}

// Sizes of an expert layer: SGEMM_OK, or what is wrong with them.
static int moe_sizes(int tokens, int hidden, int inner, int experts, int top, int type) {
    if (tokens < 0 || tokens > SGEMM_MX4_MAX_TOKENS || experts < 1 || experts > SGEMM_MX4_MAX_EXPERTS || top < 1 ||
        top > experts || top > SGEMM_MX4_MAX_TOP || hidden < 1 || inner < 1 ||
        (int64_t)experts * 2 * inner > SGEMM_MX4_MAX_DIM || (int64_t)experts * hidden > SGEMM_MX4_MAX_DIM)
        return SGEMM_ERR_SHAPE;
    return known_type(type) ? SGEMM_OK : SGEMM_ERR_CONFIG;
}

SGEMM_API int sgemm_f32_mx4_moe_scratch(int tokens, int hidden, int inner, int experts, int top, int type,
                                        long long *bytes) {
    const int status = moe_sizes(tokens, hidden, inner, experts, top, type);
    if (status != SGEMM_OK) return status;
    if (!bytes) return SGEMM_ERR_NULL;
    *bytes = mx4_moe_scratch(tokens, hidden, inner, experts, top);
    return SGEMM_OK;
}

SGEMM_API int sgemm_f32_mx4_moe(int tokens, int hidden, int inner, int experts, int top, int norm, int type, const void *X,
                                int ldx, const void *router, int ldr, const void *up, const void *sup, const void *down,
                                const void *sdown, void *Y, int ldy, void *scratch, long long scratch_bytes,
                                hipStream_t stream) {
    int status = moe_sizes(tokens, hidden, inner, experts, top, type);
    if (status != SGEMM_OK) return status;
    if (norm != 0 && norm != 1) return SGEMM_ERR_CONFIG;
    if (tokens == 0) return SGEMM_OK;
    if (ldx < hidden || ldr < hidden || ldy < hidden) return SGEMM_ERR_LD;
    const int64_t need = mx4_moe_scratch(tokens, hidden, inner, experts, top);
    const int ur = experts * 2 * inner, dr = experts * hidden;
    const Span spans[] = {floats(X, tokens, hidden, ldx, type, false), floats(router, experts, hidden, ldr, type, false),
                          codes(up, ur, hidden, false), scales(sup, ur, hidden, false),
                          codes(down, dr, inner, false), scales(sdown, dr, inner, false),
                          floats(Y, tokens, hidden, ldy, type, true), Span{scratch, need, 256, true}};
    if (scratch && scratch_bytes < need) return SGEMM_ERR_SCRATCH;
    int dev = 0;
    if ((status = check_spans(spans, &dev)) != SGEMM_OK) return status;
    return done(launch_mx4_moe({X, router, ldx, ldr, (const uint8_t *)up, (const uint8_t *)sup, (const uint8_t *)down,
                                (const uint8_t *)sdown, tokens, hidden, inner, experts, top, norm, type, Y, ldy,
                                (char *)scratch}, stream));
}
