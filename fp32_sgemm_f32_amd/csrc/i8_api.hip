// C entry points of the 8-bit integer operators (declared in
// include/sgemm_f32.h): argument checks, then one launcher each.
#include <hip/hip_runtime_api.h>

#include "checks.h"
#include "i8.h"

namespace sgemm {
namespace {

// At most 2^34 values: 32-bit counts of threads hold in every launch.
bool size_ok(int rows, int cols) {
    return rows >= 0 && rows <= SGEMM_I8_MAX_DIM && cols >= 0 && cols <= SGEMM_I8_MAX_DIM &&
           rows * i8_ld(cols) <= SGEMM_I8_MAX_VALUES;
}
bool group_ok(int group) { return group == 0 || group == SGEMM_I8_GROUP; }
int64_t values_bytes(int rows, int cols) { return rows * i8_ld(cols); }
int64_t scales_bytes(int rows, int cols, int group) { return group ? rows * (i8_ld(cols) / 128) * 4 : cols > 0 ? (int64_t)rows * 4 : 0; }

Span values(const void *p, int rows, int cols, bool out) { return Span{p, values_bytes(rows, cols), 16, out}; }
Span scales(const void *p, int rows, int cols, int group, bool out) { return Span{p, scales_bytes(rows, cols, group), 4, out}; }

int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

}  // namespace
}  // namespace sgemm

using namespace sgemm;

SGEMM_API int sgemm_f32_i8_bytes(int rows, int cols, int group, long long *values_out, long long *scales_out) {
    if (!size_ok(rows, cols)) return SGEMM_ERR_SHAPE;
    if (!group_ok(group)) return SGEMM_ERR_CONFIG;
    if (values_out) *values_out = values_bytes(rows, cols);
    if (scales_out) *scales_out = scales_bytes(rows, cols, group);
    return SGEMM_OK;
}

SGEMM_API int sgemm_f32_i8_quantize_scratch(int trans, int rows, int cols, long long *bytes) {
    if (!size_ok(rows, cols) || !size_ok(cols, rows)) return SGEMM_ERR_SHAPE;
    if (trans != 0 && trans != 1) return SGEMM_ERR_CONFIG;
    if (!bytes) return SGEMM_ERR_NULL;
    *bytes = trans ? i8_part_bytes(cols, rows) : 0;
    return SGEMM_OK;
}

SGEMM_API int sgemm_f32_i8_quantize(int trans, int rows, int cols, int group, int type, const void *X, int ldx, void *q, void *s,
                                    void *scratch, long long scratch_bytes, hipStream_t stream) {
    if (!size_ok(rows, cols) || (trans && !size_ok(cols, rows))) return SGEMM_ERR_SHAPE;
    if (!known_type(type) || !group_ok(group) || (trans != 0 && trans != 1) || (trans && group)) return SGEMM_ERR_CONFIG;
    if (rows == 0 || cols == 0) return SGEMM_OK;
    if (ldx < (trans ? rows : cols)) return SGEMM_ERR_LD;
    const int64_t need = trans ? i8_part_bytes(cols, rows) : 0;
    if (need > 0 && scratch && scratch_bytes < need) return SGEMM_ERR_SCRATCH;
    const Span spans[] = {floats(X, trans ? cols : rows, trans ? rows : cols, ldx, type, false), values(q, rows, cols, true),
                          scales(s, rows, cols, group, true), Span{scratch, need, 256, true}};
    int dev = 0;
    const int status = check_spans(spans, &dev);
    if (status != SGEMM_OK) return status;
    if (trans) return done(launch_i8_cols({X, ldx, cols, rows, type, nullptr, (uint32_t *)scratch, (int8_t *)q, (float *)s}, stream));
    if (group) return done(launch_i8_groups({X, ldx, rows, cols, type, (int8_t *)q, (float *)s}, stream));
    return done(launch_i8_rows({X, ldx, rows, cols, type, (int8_t *)q, (float *)s}, stream));
}

SGEMM_API int sgemm_f32_i8_dequantize(int rows, int cols, int group, const void *q, const void *s, int type, void *Y, int ldy,
                                      hipStream_t stream) {
    if (!size_ok(rows, cols)) return SGEMM_ERR_SHAPE;
    if (!known_type(type) || !group_ok(group)) return SGEMM_ERR_CONFIG;
    if (rows == 0 || cols == 0) return SGEMM_OK;
    if (ldy < cols) return SGEMM_ERR_LD;
    const Span spans[] = {values(q, rows, cols, false), scales(s, rows, cols, group, false), floats(Y, rows, cols, ldy, type, true)};
    int dev = 0;
    const int status = check_spans(spans, &dev);
    if (status != SGEMM_OK) return status;
    return done(launch_i8_back({(const int8_t *)q, (const float *)s, rows, cols, group, type, Y, ldy}, stream));
}

SGEMM_API int sgemm_f32_i8_gemm(int M, int N, int K, float alpha, const void *a, const void *sa, const void *b, const void *sb,
                                float beta, int type, void *C, int ldc, hipStream_t stream) {
    if (!size_ok(M, K) || !size_ok(N, K) || K > SGEMM_I8_MAX_SUM) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (ldc < N) return SGEMM_ERR_LD;
    const int k = alpha == 0.0f ? 0 : K;   // nothing of A and B is read then
    if (K == 0) alpha = 0.0f;              // an empty sum stays zero whatever alpha
    const Span spans[] = {values(a, M, k, false), scales(sa, M, k, 0, false), values(b, N, k, false), scales(sb, N, k, 0, false),
                          floats(C, M, N, ldc, type, true)};
    int dev = 0, cus = 0;
    int status = check_spans(spans, &dev);
    if (status == SGEMM_OK) status = compute_units(dev, &cus);
    if (status != SGEMM_OK) return status;
    return done(launch_i8_gemm({(const int8_t *)a, k > 0 ? (const float *)sa : nullptr, (const int8_t *)b,
                                k > 0 ? (const float *)sb : nullptr, M, N, k, type, 0, 1, alpha, beta, C, ldc}, cus, stream));
}

// Scratch memory of a product with float rows: their 8-bit form, where a kernel of its own makes it.
static int64_t linear_scratch(int M, int N, int K) {
    return K > 0 && !i8_thin_takes_floats(M, N, K) ? up256(values_bytes(M, K)) + up256((int64_t)M * 4) : 0;
}

SGEMM_API int sgemm_f32_i8_linear_scratch(int M, int N, int K, int type, long long *bytes) {
    if (!size_ok(M, K) || !size_ok(N, K) || K > SGEMM_I8_MAX_SUM) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (!bytes) return SGEMM_ERR_NULL;
    *bytes = linear_scratch(M, N, K);
    return SGEMM_OK;
}

SGEMM_API int sgemm_f32_i8_linear(int M, int N, int K, int type, const void *X, int ldx, const void *w, const void *sw, void *Y,
                                  int ldy, void *scratch, long long scratch_bytes, hipStream_t stream) {
    if (!size_ok(M, K) || !size_ok(N, K) || K > SGEMM_I8_MAX_SUM) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (ldx < K || ldy < N) return SGEMM_ERR_LD;
    const int64_t need = linear_scratch(M, N, K);
    if (scratch && scratch_bytes < need) return SGEMM_ERR_SCRATCH;
    const Span spans[] = {floats(X, M, K, ldx, type, false), values(w, N, K, false), scales(sw, N, K, 0, false),
                          floats(Y, M, N, ldy, type, true), Span{scratch, need, 256, true}};
    int dev = 0, cus = 0;
    int status = check_spans(spans, &dev);
    if (status == SGEMM_OK) status = compute_units(dev, &cus);
    if (status != SGEMM_OK) return status;
    if (K > 0 && need == 0)
        return done(launch_i8_thin({nullptr, nullptr, (const int8_t *)w, (const float *)sw, M, N, K, type, 0, 1, 1.0f, 0.0f, Y, ldy}, X, ldx,
                                   cus, stream));
    int8_t *q = (int8_t *)scratch;
    float *s = K > 0 ? (float *)(q + up256(values_bytes(M, K))) : nullptr;
    const hipError_t e = K > 0 ? launch_i8_rows({X, ldx, M, K, type, q, s}, stream) : hipSuccess;
    if (e != hipSuccess) return done(e);
    return done(launch_i8_gemm({q, s, (const int8_t *)w, K > 0 ? (const float *)sw : nullptr, M, N, K, type, 0, 1, K > 0 ? 1.0f : 0.0f,
                                0.0f, Y, ldy}, cus, stream));
}

// A training step's sizes: each is the length of a sum, and a side of what is quantised both ways.
static bool train_ok(int M, int N, int K) {
    return M <= SGEMM_I8_MAX_SUM && N <= SGEMM_I8_MAX_SUM && K <= SGEMM_I8_MAX_SUM && size_ok(M, K) && size_ok(N, K) && size_ok(M, N) &&
           size_ok(N, M);
}

SGEMM_API int sgemm_f32_i8_train_forward(int M, int N, int K, int type, const void *X, int ldx, int type_w, const void *W, int ldw,
                                         void *Y, int ldy, void *xq, void *sx, void *wq, void *sw, hipStream_t stream) {
    if (!train_ok(M, N, K)) return SGEMM_ERR_SHAPE;
    if (!known_type(type) || !known_type(type_w)) return SGEMM_ERR_CONFIG;
    const bool x = M > 0 && K > 0, w = N > 0 && K > 0, y = M > 0 && N > 0;
    if ((x && ldx < K) || (w && ldw < K) || (y && ldy < N)) return SGEMM_ERR_LD;
    const Span spans[] = {floats(X, M, K, ldx, type, false), floats(W, N, K, ldw, type_w, false), floats(Y, M, N, ldy, type, true),
                          values(xq, M, K, true), scales(sx, M, K, 0, true), values(wq, N, K, true), scales(sw, N, K, 0, true)};
    int dev = 0, cus = 0;
    int status = check_spans(spans, &dev);
    if (status == SGEMM_OK) status = compute_units(dev, &cus);
    if (status != SGEMM_OK) return status;
    const I8RowsJob jx{X, ldx, M, K, type, (int8_t *)xq, (float *)sx}, jw{W, ldw, N, K, type_w, (int8_t *)wq, (float *)sw};
    hipError_t e = hipSuccess;
    if (x && w && type == type_w) {
        e = launch_i8_rows_two(jx, jw, stream);
    } else {
        if (x) e = launch_i8_rows(jx, stream);
        if (w && e == hipSuccess) e = launch_i8_rows(jw, stream);
    }
    if (e == hipSuccess && y)
        e = launch_i8_gemm({(const int8_t *)xq, K > 0 ? (const float *)sx : nullptr, (const int8_t *)wq, K > 0 ? (const float *)sw : nullptr,
                            M, N, K, type, 0, 1, K > 0 ? 1.0f : 0.0f, 0.0f, Y, ldy}, cus, stream);
    return done(e);
}

// Scratch memory of the backward pass: dY by row, by column in two pieces, the
// scales of both, and the columns' largest magnitudes.
namespace {
struct Back {
    int64_t d, sd, t, st, part, bytes;
};
Back back_layout(int M, int N) {
    Back b;
    int64_t at = 0;
    const auto take = [&](int64_t n) { const int64_t here = at; at += up256(n); return here; };
    b.d = take(values_bytes(M, N));
    b.sd = take((int64_t)M * 4);
    b.t = take(i8_piece_rows(N) * i8_ld(M));
    b.st = take((int64_t)N * 4);
    b.part = take(i8_both_part_bytes(M, N));
    b.bytes = M > 0 && N > 0 ? at : 0;
    return b;
}
}  // namespace

SGEMM_API int sgemm_f32_i8_train_scratch(int M, int N, int K, long long *bytes) {
    if (!train_ok(M, N, K)) return SGEMM_ERR_SHAPE;
    if (!bytes) return SGEMM_ERR_NULL;
    *bytes = back_layout(M, N).bytes;
    return SGEMM_OK;
}

SGEMM_API int sgemm_f32_i8_train_backward(int M, int N, int K, int type, const void *dY, int ldd, const void *xq, const void *sx,
                                          const void *wq, const void *sw, void *dX, int lddx, float beta, void *dW, int lddw,
                                          void *scratch, long long scratch_bytes, hipStream_t stream) {
    if (!train_ok(M, N, K)) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    const bool d = M > 0 && N > 0 && K > 0, x = M > 0 && K > 0, w = N > 0 && K > 0;
    if ((d && ldd < N) || (x && lddx < K) || (w && lddw < K)) return SGEMM_ERR_LD;
    const Back at = back_layout(M, N);
    if (scratch && scratch_bytes < at.bytes) return SGEMM_ERR_SCRATCH;
    const Span spans[] = {floats(dY, d ? M : 0, N, ldd, type, false), values(xq, M, K, false), scales(sx, M, K, 0, false),
                          values(wq, N, K, false), scales(sw, N, K, 0, false), floats(dX, M, K, lddx, type, true),
                          floats(dW, N, K, lddw, SGEMM_TYPE_F32, true), Span{scratch, at.bytes, 256, true}};
    int dev = 0, cus = 0;
    int status = check_spans(spans, &dev);
    if (status == SGEMM_OK) status = compute_units(dev, &cus);
    if (status != SGEMM_OK) return status;
    char *p = (char *)scratch;
    int8_t *dq = (int8_t *)(p + at.d), *tq = (int8_t *)(p + at.t);
    float *sd = (float *)(p + at.sd), *st = (float *)(p + at.st);
    hipError_t e = hipSuccess;
    if (d)
        e = launch_i8_both({dY, ldd, M, N, type, (const float *)sw, (const float *)sx, (uint32_t *)(p + at.part), dq, sd, tq, st}, stream);
    const I8GemmJob gx{dq, N > 0 ? sd : nullptr, (const int8_t *)wq, nullptr, M, K, N, type, 1, 1, N > 0 ? 1.0f : 0.0f, 0.0f, dX, lddx};
    const I8GemmJob gw{tq, M > 0 ? st : nullptr, (const int8_t *)xq, nullptr, N, K, M, SGEMM_TYPE_F32, 1, 2, M > 0 ? 1.0f : 0.0f, beta, dW, lddw};
    if (e == hipSuccess) e = x && w ? launch_i8_gemm_two(gx, gw, cus, stream)
                             : x    ? launch_i8_gemm(gx, cus, stream)
                             : w    ? launch_i8_gemm(gw, cus, stream)
                                    : hipSuccess;
    return done(e);
}

SGEMM_API int sgemm_f32_i8_swiglu_forward(int rows, int inner, int type, const void *GU, int ldx, void *H, int ldh, void *gq, void *gs,
                                          void *uq, void *us, hipStream_t stream) {
    if (!size_ok(rows, inner) || inner > SGEMM_I8_MAX_DIM / 2) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (rows == 0 || inner == 0) return SGEMM_OK;
    if (ldx < 2 * inner || ldh < inner) return SGEMM_ERR_LD;
    const Span spans[] = {floats(GU, rows, 2 * inner, ldx, type, false), floats(H, rows, inner, ldh, type, true),
                          values(gq, rows, inner, true), scales(gs, rows, inner, SGEMM_I8_GROUP, true),
                          values(uq, rows, inner, true), scales(us, rows, inner, SGEMM_I8_GROUP, true)};
    int dev = 0;
    const int status = check_spans(spans, &dev);
    if (status != SGEMM_OK) return status;
    return done(launch_i8_swiglu_forward({GU, ldx, rows, inner, type, (int8_t *)gq, (float *)gs, (int8_t *)uq, (float *)us, H, ldh}, stream));
}

SGEMM_API int sgemm_f32_i8_swiglu_backward(int rows, int inner, int type, const void *dH, int ldd, const void *gq, const void *gs,
                                           const void *uq, const void *us, void *dGU, int ldy, hipStream_t stream) {
    if (!size_ok(rows, inner) || inner > SGEMM_I8_MAX_DIM / 2) return SGEMM_ERR_SHAPE;
    if (!known_type(type)) return SGEMM_ERR_CONFIG;
    if (rows == 0 || inner == 0) return SGEMM_OK;
    if (ldd < inner || ldy < 2 * inner) return SGEMM_ERR_LD;
    const Span spans[] = {floats(dH, rows, inner, ldd, type, false), values(gq, rows, inner, false),
                          scales(gs, rows, inner, SGEMM_I8_GROUP, false), values(uq, rows, inner, false),
                          scales(us, rows, inner, SGEMM_I8_GROUP, false), floats(dGU, rows, 2 * inner, ldy, type, true)};
    int dev = 0;
    const int status = check_spans(spans, &dev);
    if (status != SGEMM_OK) return status;
    return done(launch_i8_swiglu_backward({dH, ldd, rows, inner, type, (int8_t *)gq, (float *)gs, (int8_t *)uq, (float *)us, dGU, ldy}, stream));
}
