// gq_act_api.cu -- host side of the activation checkpoints' entry points (include/gq.h): argument
// checks and kernel selection.
#include <cstdint>

#include "gq_act.h"
#include "gq_check.h"

namespace {

using namespace gq;

gq_status_t act_check(int dtype, int64_t rows, int64_t cols)
{
    if (!elem_size(dtype) || !shape_ok(rows, cols)) return GQ_ERR_INVALID;
    return GQ_OK;
}

}  // namespace

extern "C" {

gq_status_t gq_act_layout(int64_t rows, int64_t cols, size_t *bytes, size_t *codes_off, size_t *exps_off)
{
    if (!shape_ok(rows, cols)) return GQ_ERR_INVALID;
    const gq::CkptLayout l = gq::ckpt_layout(rows, cols);
    if (bytes) *bytes = l.bytes;
    if (codes_off) *codes_off = 0;
    if (exps_off) *exps_off = l.exps_off;
    return GQ_OK;
}

gq_status_t gq_act_pack(int dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride, void *ckpt, void *stream)
{
    Range range("gq_act_pack");
    const gq_status_t st = act_check(dtype, rows, cols);
    if (st != GQ_OK) return st;
    if (rows == 0) return GQ_OK;
    if (!in_ok(x, rows, x_stride) || !ckpt || !aligned(ckpt, 16)) return GQ_ERR_INVALID;
    const Region w[] = {region(ckpt, gq::ckpt_layout(rows, cols).bytes)};
    const Region r[] = {region(x, rows, cols, x_stride, elem_size(dtype))};
    if (any_overlap(w, 1, r, 1)) return GQ_ERR_INVALID;
    const gq::ActArgs a = {dtype, 0, rows, cols, {x, x_stride}, {nullptr, 0}, ckpt};
    return from_cuda(gq::launch_act(gq::kPack, a, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_act_unpack(int dtype, int64_t rows, int64_t cols, const void *ckpt, void *x, int64_t x_stride, void *stream)
{
    Range range("gq_act_unpack");
    const gq_status_t st = act_check(dtype, rows, cols);
    if (st != GQ_OK) return st;
    if (rows == 0) return GQ_OK;
    if (!out_ok(x, rows, cols, x_stride) || !ckpt || !aligned(ckpt, 16)) return GQ_ERR_INVALID;
    const Region w[] = {region(x, rows, cols, x_stride, elem_size(dtype))};
    const Region r[] = {region(ckpt, gq::ckpt_layout(rows, cols).bytes)};
    if (any_overlap(w, 1, r, 1)) return GQ_ERR_INVALID;
    const gq::ActArgs a = {dtype, 0, rows, cols, {nullptr, 0}, {x, x_stride}, const_cast<void *>(ckpt)};
    return from_cuda(gq::launch_act(gq::kUnpack, a, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_act_fn_forward(int kind, int dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride, void *y,
                              int64_t y_stride, void *ckpt, void *stream)
{
    Range range("gq_act_fn_forward");
    if (kind < GQ_FN_GELU || kind > GQ_FN_SILU) return GQ_ERR_INVALID;
    const gq_status_t st = act_check(dtype, rows, cols);
    if (st != GQ_OK) return st;
    if (rows == 0) return GQ_OK;
    if (!in_ok(x, rows, x_stride) || !out_ok(y, rows, cols, y_stride) || !aligned(ckpt, 16)) return GQ_ERR_INVALID;
    const int size = elem_size(dtype);
    const Region w[] = {region(y, rows, cols, y_stride, size), region(ckpt, gq::ckpt_layout(rows, cols).bytes)};
    const Region r[] = {region(x, rows, cols, x_stride, size)};
    if (any_overlap(w, 2, r, 1)) return GQ_ERR_INVALID;
    const gq::ActArgs a = {dtype, kind, rows, cols, {x, x_stride}, {y, y_stride}, ckpt};
    return from_cuda(gq::launch_act(ckpt ? gq::kForwardKeep : gq::kForward, a, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_act_fn_backward(int kind, int dtype, int64_t rows, int64_t cols, const void *ckpt, const void *dy,
                               int64_t dy_stride, void *dx, int64_t dx_stride, void *stream)
{
    Range range("gq_act_fn_backward");
    if (kind < GQ_FN_GELU || kind > GQ_FN_SILU) return GQ_ERR_INVALID;
    const gq_status_t st = act_check(dtype, rows, cols);
    if (st != GQ_OK) return st;
    if (rows == 0) return GQ_OK;
    if (!in_ok(dy, rows, dy_stride) || !out_ok(dx, rows, cols, dx_stride) || !ckpt || !aligned(ckpt, 16))
        return GQ_ERR_INVALID;
    const int size = elem_size(dtype);
    const Region w[] = {region(dx, rows, cols, dx_stride, size)};
    const Region r[] = {region(dy, rows, cols, dy_stride, size), region(ckpt, gq::ckpt_layout(rows, cols).bytes)};
    if (any_overlap(w, 1, r, 2)) return GQ_ERR_INVALID;
    const gq::ActArgs a = {dtype, kind, rows, cols, {dy, dy_stride}, {dx, dx_stride}, const_cast<void *>(ckpt)};
    return from_cuda(gq::launch_act(gq::kBackward, a, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_act_weight_grad_workspace(int dtype, int64_t tokens, int64_t in, int64_t out, int64_t dy_stride, int bias,
                                         size_t *bytes)
{
    if (!elem_size(dtype) || !shape_ok(tokens, in) || !shape_ok(tokens, out) || !bytes) return GQ_ERR_INVALID;
    *bytes = gq::wgrad_workspace(dtype, tokens, in, out, dy_stride, bias != 0);
    return GQ_OK;
}

gq_status_t gq_act_weight_grad(int dtype, int64_t tokens, int64_t in, int64_t out, const void *ckpt, const void *dy,
                               int64_t dy_stride, float *dw, int64_t dw_stride, float *db, int accumulate, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    Range range("gq_act_weight_grad");
    if (!elem_size(dtype) || !shape_ok(tokens, in) || !shape_ok(tokens, out)) return GQ_ERR_INVALID;
    if (accumulate != 0 && accumulate != 1) return GQ_ERR_INVALID;
    if (!dw || !aligned(dw, 4) || !aligned(db, 4) || (out > 1 && (dw_stride < in || dw_stride > (int64_t(1) << 40))))
        return GQ_ERR_INVALID;
    if (tokens > 0 && (!in_ok(dy, tokens, dy_stride) || !ckpt || !aligned(ckpt, 16))) return GQ_ERR_INVALID;
    const size_t need = gq::wgrad_workspace(dtype, tokens, in, out, dy_stride, db != nullptr);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return GQ_ERR_INVALID;
    const Region w[] = {region(dw, out, in, dw_stride, 4), region(db, (size_t)out * 4), region(workspace, need)};
    const Region r[] = {region(dy, tokens, out, dy_stride, elem_size(dtype)),
                        region(ckpt, gq::ckpt_layout(tokens, in).bytes)};
    if (any_overlap(w, 3, r, 2)) return GQ_ERR_INVALID;
    const gq::WgradArgs a = {dtype, tokens, in, out, ckpt, {dy, dy_stride}, dw, dw_stride, db, accumulate,
                             static_cast<unsigned char *>(workspace)};
    return from_cuda(gq::launch_wgrad(a, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_layer_norm_forward(int dtype, int param_dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride,
                                  const void *gamma, const void *beta, float eps, void *y, int64_t y_stride, float *mean,
                                  float *rstd, void *ckpt, void *stream)
{
    Range range("gq_layer_norm_forward");
    const gq_status_t st = act_check(dtype, rows, cols);
    if (st != GQ_OK) return st;
    if (param_dtype != dtype && param_dtype != GQ_FLOAT32) return GQ_ERR_INVALID;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    const int psize = elem_size(param_dtype), size = elem_size(dtype);
    if (!in_ok(x, rows, x_stride) || !out_ok(y, rows, cols, y_stride) || !mean || !rstd || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(ckpt, 16) || !aligned(gamma, (uintptr_t)psize) || !aligned(beta, (uintptr_t)psize))
        return GQ_ERR_INVALID;
    const Region w[] = {region(y, rows, cols, y_stride, size), region(mean, (size_t)rows * 4),
                        region(rstd, (size_t)rows * 4), region(ckpt, gq::ckpt_layout(rows, cols).bytes)};
    const Region r[] = {region(x, rows, cols, x_stride, size), region(gamma, (size_t)(cols * psize)),
                        region(beta, (size_t)(cols * psize))};
    if (any_overlap(w, 4, r, 3)) return GQ_ERR_INVALID;
    gq::NormArgs a = {};
    a.dtype = dtype;
    a.param_dtype = param_dtype;
    a.rows = rows;
    a.cols = cols;
    a.x = {x, x_stride};
    a.y = {y, y_stride};
    a.ckpt = ckpt;
    a.gamma = gamma;
    a.beta = beta;
    a.mean = mean;
    a.rstd = rstd;
    a.eps = eps;
    return from_cuda(gq::launch_norm_forward(a, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_layer_norm_workspace(int64_t rows, int64_t cols, size_t *bytes)
{
    if (!shape_ok(rows, cols) || !bytes) return GQ_ERR_INVALID;
    *bytes = (size_t)gq::norm_parts(rows, cols) * (size_t)cols * 2 * sizeof(float);
    return GQ_OK;
}

gq_status_t gq_layer_norm_backward(int dtype, int param_dtype, int64_t rows, int64_t cols, const void *dy,
                                   int64_t dy_stride, const void *x, int64_t x_stride, const void *ckpt, const void *gamma,
                                   const float *mean, const float *rstd, void *dx, int64_t dx_stride, float *dgamma,
                                   float *dbeta, int accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    Range range("gq_layer_norm_backward");
    const gq_status_t st = act_check(dtype, rows, cols);
    if (st != GQ_OK) return st;
    if (param_dtype != dtype && param_dtype != GQ_FLOAT32) return GQ_ERR_INVALID;
    if (accumulate != 0 && accumulate != 1) return GQ_ERR_INVALID;
    const int psize = elem_size(param_dtype), size = elem_size(dtype);
    if (!aligned(dgamma, 4) || !aligned(dbeta, 4) || !aligned(gamma, (uintptr_t)psize)) return GQ_ERR_INVALID;
    if (rows > 0) {
        if ((x != nullptr) == (ckpt != nullptr)) return GQ_ERR_INVALID;
        if (x && !in_ok(x, rows, x_stride)) return GQ_ERR_INVALID;
        if (!aligned(ckpt, 16) || !in_ok(dy, rows, dy_stride) || !out_ok(dx, rows, cols, dx_stride) || !mean || !rstd ||
            !aligned(mean, 4) || !aligned(rstd, 4))
            return GQ_ERR_INVALID;
    }
    const bool grads = dgamma || dbeta;
    const size_t need = grads ? (size_t)gq::norm_parts(rows, cols) * (size_t)cols * 2 * sizeof(float) : 0;
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return GQ_ERR_INVALID;
    const Region w[] = {region(dx, rows, cols, dx_stride, size), region(dgamma, (size_t)cols * 4),
                        region(dbeta, (size_t)cols * 4), region(workspace, need)};
    const Region r[] = {region(dy, rows, cols, dy_stride, size),        region(x, rows, cols, x_stride, size),
                        region(ckpt, gq::ckpt_layout(rows, cols).bytes), region(gamma, (size_t)(cols * psize)),
                        region(mean, (size_t)rows * 4),                  region(rstd, (size_t)rows * 4)};
    if (any_overlap(w, 4, r, 6)) return GQ_ERR_INVALID;
    gq::NormArgs a = {};
    a.dtype = dtype;
    a.param_dtype = param_dtype;
    a.rows = rows;
    a.cols = cols;
    a.x = {x, x_stride};
    a.y = {dx, dx_stride};
    a.dy = {dy, dy_stride};
    a.ckpt = const_cast<void *>(ckpt);
    a.gamma = gamma;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.accumulate = accumulate;
    a.parts = grads ? static_cast<float *>(workspace) : nullptr;
    return from_cuda(gq::launch_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
