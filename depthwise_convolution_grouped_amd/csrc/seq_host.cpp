// Host side of the sequence operators of include/gconv.h: checks of the
// descriptors and pointers, all before any HIP call, and the calls of the
// kernels' launchers.
#include <math.h>

#include "seq_internal.h"

#define GCONV_API extern "C" __attribute__((visibility("default")))

namespace gconv {
namespace {

constexpr int64_t kMost = INT32_MAX - 1023;    // an extent: the kernels' int indices run past it by up to a block
constexpr int64_t kMostStride = 1ll << 40;     // a stride, in elements
constexpr int64_t kMostK = 131071;             // 2^31 / (128 * 128), rounded down to stay below it

uintptr_t elem(int dtype) { return dtype == GCONV_F32 ? 4 : 2; }
bool dtype_ok(int t) { return t == GCONV_F32 || t == GCONV_F16 || t == GCONV_BF16; }
bool extent_ok(int64_t v, int64_t least) { return v >= least && v <= kMost; }

// Rows of D channels with [0] the batch and [1] the time stride.
bool read_ok(const int64_t st[2])
{
    return st[0] >= 0 && st[1] >= 0 && st[0] <= kMostStride && st[1] <= kMostStride;
}

// No two elements of an output at the same place: the smaller of the two
// strides passes a row, the larger one passes all rows of the other axis.
bool write_ok(const int64_t st[2], int64_t B, int64_t L, int64_t D)
{
    if (!read_ok(st)) return false;
    if (B == 0 || L == 0) return true;   // nothing is written
    const bool b = B > 1, t = L > 1;
    if (b && t) {
        const int in = st[0] <= st[1] ? 0 : 1;
        const int64_t n = in == 0 ? B : L;
        return st[in] >= D && st[1 - in] / st[in] >= n - 1 && st[1 - in] - (n - 1) * st[in] >= D;
    }
    if (b) return st[0] >= D;
    return !t || st[1] >= D;
}

int check(const gconv_glr_desc *d, bool backward)
{
    if (!d) return GCONV_ERR_NULL_PTR;
    if (!dtype_ok(d->dtype) || !(d->c > 0.0f) || !isfinite(d->c)) return GCONV_ERR_BAD_DESC;
    if (d->B < 0 || d->L < 0 || d->D < 1) return GCONV_ERR_BAD_DESC;
    if (!read_ok(d->x_stride) || !read_ok(d->r_stride) || !read_ok(d->i_stride)) return GCONV_ERR_BAD_DESC;
    if (!extent_ok(d->B, 0) || !extent_ok(d->L, 0) || !extent_ok(d->D, 1)) return GCONV_ERR_TOO_LARGE;
    if (backward) {
        if (!read_ok(d->y_stride)) return GCONV_ERR_BAD_DESC;
        for (const int64_t *st : {d->dx_stride, d->dr_stride, d->di_stride})
            if (!write_ok(st, d->B, d->L, d->D)) return GCONV_ERR_BAD_DESC;
    } else if (!write_ok(d->y_stride, d->B, d->L, d->D)) {
        return GCONV_ERR_BAD_DESC;
    }
    return glr::fits(*d, backward) ? GCONV_OK : GCONV_ERR_TOO_LARGE;
}

int check(const gconv_q8_desc *d, const void *x, const void *residual, const void *weight, const void *q,
          const void *scale, const void *sum, bool norm)
{
    if (!d) return GCONV_ERR_NULL_PTR;
    if (!dtype_ok(d->dtype) || d->M < 0 || d->D < 1) return GCONV_ERR_BAD_DESC;
    if (norm && (!(d->eps >= 0.0f) || !isfinite(d->eps))) return GCONV_ERR_BAD_DESC;
    if (!extent_ok(d->M, 0) || !extent_ok(d->D, 1)) return GCONV_ERR_TOO_LARGE;
    if (d->x_stride < 0 || d->x_stride > kMostStride) return GCONV_ERR_BAD_DESC;
    if (residual && (d->residual_stride < 0 || d->residual_stride > kMostStride)) return GCONV_ERR_BAD_DESC;
    if (d->M > 1 && (d->q_stride < d->D || (sum && d->sum_stride < d->D))) return GCONV_ERR_BAD_DESC;
    if (d->q_stride < 0 || d->q_stride > kMostStride) return GCONV_ERR_BAD_DESC;
    if (sum && (!residual || d->sum_stride < 0 || d->sum_stride > kMostStride)) return GCONV_ERR_BAD_DESC;
    if (d->M == 0) return GCONV_OK;
    if (!x || !q || !scale || (norm && !weight)) return GCONV_ERR_NULL_PTR;
    const uintptr_t e = elem(d->dtype);
    if (!on(x, e) || !on(residual, e) || !on(sum, e) || !on(weight, 4) || !on(scale, 4)) return GCONV_ERR_MISALIGNED;
    return GCONV_OK;
}

int check(const gconv_mm_q8_desc *d)
{
    if (!d) return GCONV_ERR_NULL_PTR;
    if (!dtype_ok(d->dtype) || d->reserved != 0 || d->M < 0 || d->N < 1 || d->K < 1) return GCONV_ERR_BAD_DESC;
    if (!extent_ok(d->M, 0) || !extent_ok(d->N, 1) || d->K > kMostK) return GCONV_ERR_TOO_LARGE;
    if (d->a_stride < 0 || d->a_stride > kMostStride || d->w_stride < 0 || d->w_stride > kMostStride)
        return GCONV_ERR_BAD_DESC;
    if (d->y_stride < 0 || d->y_stride > kMostStride || (d->M > 1 && d->y_stride < d->N)) return GCONV_ERR_BAD_DESC;
    return GCONV_OK;
}

int status(hipError_t e) { return e == hipSuccess ? GCONV_OK : GCONV_ERR_LAUNCH; }

}  // namespace
}  // namespace gconv

using namespace gconv;

GCONV_API int gconv_glr_fwd_workspace(const gconv_glr_desc *d, size_t *bytes)
{
    if (!bytes) return GCONV_ERR_NULL_PTR;
    const int rc = check(d, false);
    if (rc != GCONV_OK) return rc;
    *bytes = glr::fwd_workspace(*d);
    return GCONV_OK;
}

GCONV_API int gconv_glr_fwd(const gconv_glr_desc *d, const void *x, const void *r, const void *i,
                            const float *lambda, const float *h0, const int32_t *lengths, void *y, float *h_last,
                            float *states, void *workspace, size_t workspace_bytes, void *stream)
{
    const int rc = check(d, false);
    if (rc != GCONV_OK) return rc;
    if (d->B == 0) return GCONV_OK;
    if (!lambda || (d->L > 0 && (!x || !r || !i || !y))) return GCONV_ERR_NULL_PTR;
    const uintptr_t e = elem(d->dtype);
    if (!on(x, e) || !on(r, e) || !on(i, e) || !on(y, e) || !on(lambda, 4) || !on(h0, 4) || !on(lengths, 4) ||
        !on(h_last, 4) || !on(states, 4) || !on(workspace, 4))
        return GCONV_ERR_MISALIGNED;
    const glr::Fwd a{x, r, i, lambda, h0, lengths, y, h_last, states, (float *)workspace};
    return status(glr::fwd(*d, a, workspace ? workspace_bytes : 0, (hipStream_t)stream));
}

GCONV_API int gconv_glr_bwd_workspace(const gconv_glr_desc *d, size_t *bytes, size_t *min_bytes)
{
    const int rc = check(d, true);
    if (rc != GCONV_OK) return rc;
    if (bytes) *bytes = glr::bwd_workspace(*d);
    if (min_bytes) *min_bytes = glr::bwd_min_workspace(*d);
    return GCONV_OK;
}

GCONV_API int gconv_glr_bwd(const gconv_glr_desc *d, const void *x, const void *r, const void *i,
                            const float *lambda, const int32_t *lengths, const float *states, const void *dy,
                            const float *dh_last, void *dx, void *dr, void *di, float *dlambda, float *dh0,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    const int rc = check(d, true);
    if (rc != GCONV_OK) return rc;
    if (!lambda || !dlambda) return GCONV_ERR_NULL_PTR;
    if (d->B > 0 && d->L > 0 && (!x || !r || !i || !states || !dy || !dx || !dr || !di)) return GCONV_ERR_NULL_PTR;
    const uintptr_t e = elem(d->dtype);
    if (!on(x, e) || !on(r, e) || !on(i, e) || !on(dy, e) || !on(dx, e) || !on(dr, e) || !on(di, e) ||
        !on(lambda, 4) || !on(lengths, 4) || !on(states, 4) || !on(dh_last, 4) || !on(dlambda, 4) || !on(dh0, 4) ||
        !on(workspace, 4))
        return GCONV_ERR_MISALIGNED;
    if ((workspace ? workspace_bytes : 0) < glr::bwd_min_workspace(*d)) return GCONV_ERR_WORKSPACE;
    const glr::Bwd a{x, r, i, lambda, lengths, states, dy, dh_last, dx, dr, di, dlambda, dh0, (float *)workspace};
    return status(glr::bwd(*d, a, workspace_bytes, (hipStream_t)stream));
}

GCONV_API int gconv_rmsnorm_q8(const gconv_q8_desc *d, const void *x, const void *residual, const float *weight,
                               int8_t *q, float *scale, void *sum, void *stream)
{
    const int rc = check(d, x, residual, weight, q, scale, sum, true);
    if (rc != GCONV_OK || d->M == 0) return rc;
    return status(rowq8::run(*d, x, residual, weight, q, scale, sum, (hipStream_t)stream));
}

GCONV_API int gconv_quant_q8(const gconv_q8_desc *d, const void *x, int8_t *q, float *scale, void *stream)
{
    const int rc = check(d, x, nullptr, nullptr, q, scale, nullptr, false);
    if (rc != GCONV_OK || d->M == 0) return rc;
    return status(rowq8::run(*d, x, nullptr, nullptr, q, scale, nullptr, (hipStream_t)stream));
}

GCONV_API int gconv_matmul_q8_workspace(const gconv_mm_q8_desc *d, size_t *bytes)
{
    if (!bytes) return GCONV_ERR_NULL_PTR;
    const int rc = check(d);
    if (rc != GCONV_OK) return rc;
    *bytes = mmq8::workspace(*d);
    return GCONV_OK;
}

GCONV_API const char *gconv_matmul_q8_kernel(const gconv_mm_q8_desc *d, const void *a, const void *w,
                                             const void *workspace, size_t workspace_bytes)
{
    return check(d) == GCONV_OK ? mmq8::kernel(*d, a, w, workspace, workspace ? workspace_bytes : 0) : "";
}

GCONV_API int gconv_matmul_q8(const gconv_mm_q8_desc *d, const int8_t *a, const float *a_scale, const int8_t *w,
                              const float *w_scale, const float *bias, void *y, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    const int rc = check(d);
    if (rc != GCONV_OK || d->M == 0) return rc;
    if (!a || !a_scale || !w || !w_scale || !y) return GCONV_ERR_NULL_PTR;
    if (!on(y, elem(d->dtype)) || !on(a_scale, 4) || !on(w_scale, 4) || !on(bias, 4) || !on(workspace, 4))
        return GCONV_ERR_MISALIGNED;
    return status(mmq8::run(*d, a, a_scale, w, w_scale, bias, y, workspace, workspace ? workspace_bytes : 0,
                            (hipStream_t)stream));
}
