// block_ops.cpp -- host side of the operators around a mixer in a block:
// layer norm with dropout and residual, and dropout alone.
#include <hip/hip_runtime.h>

#include <string>

#include "host.hpp"
#include "kernels.hpp"
#include "selscan.h"

using namespace selscan::host;
using selscan::set_error;

namespace {

bool is_dtype(int32_t d) { return d == SELSCAN_F32 || d == SELSCAN_BF16; }

// The words of the generator that keep their element: floor(p 2^32) and up.
uint64_t keep_from(double p) { return (uint64_t)(p * 4294967296.0); }
float keep_scale(double p) { return p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f; }
bool is_probability(double p) { return p >= 0.0 && p <= 1.0; }   // false for NaN

selscan_status_t check_norm(const selscan_norm_shape_t* s) {
    if (!s) return set_error(SELSCAN_ERR_INVALID_ARG, "shape is NULL");
    if (s->rows < 1 || s->dim < 1) return set_error(SELSCAN_ERR_INVALID_ARG, "rows and dim must be >= 1");
    if (!is_dtype(s->in_dtype) || !is_dtype(s->res_dtype) || !is_dtype(s->out_dtype))
        return set_error(SELSCAN_ERR_UNSUPPORTED, "dtypes must be SELSCAN_F32 or SELSCAN_BF16");
    if (!(s->eps >= 0.0f)) return set_error(SELSCAN_ERR_INVALID_ARG, "eps must be >= 0");
    if (!is_probability(s->p)) return set_error(SELSCAN_ERR_INVALID_ARG, "p must be in [0, 1]");
    if (mul_checked({s->rows, s->dim, 4}) < 0 || mul_checked({s->dim, 2048, 8}) < 0)
        return set_error(SELSCAN_ERR_INVALID_ARG, "tensor sizes overflow 64-bit byte counts");
    if (s->rows > 0x7fffffff || s->dim > 0xfffffff)
        return set_error(SELSCAN_ERR_UNSUPPORTED, "layer norm supports rows < 2^31 and dim < 2^28");
    return SELSCAN_OK;
}

void fill(selscan::NormArgs& a, const selscan_norm_shape_t* s) {
    a.rows = s->rows; a.dim = s->dim; a.eps = s->eps; a.inv_dim = (float)(1.0 / (double)s->dim);
    a.seed = s->seed; a.offset = s->offset;
    a.drop = s->p > 0.0;
    a.keep_from = keep_from(s->p);
    a.keep_scale = keep_scale(s->p);
}

size_t norm_bwd_bytes(const selscan_norm_shape_t* s) {
    return align256(selscan::norm_bwd_part_bytes(s->rows, s->dim));
}

selscan_status_t launched(hipError_t e) {
    if (e != hipSuccess)
        return set_error(SELSCAN_ERR_LAUNCH, std::string("kernel launch failed: ") + hipGetErrorString(e));
    return set_error(SELSCAN_OK, "");
}

}  // namespace

extern "C" {

selscan_status_t selscan_dropout(const selscan_dropout_shape_t* s, const void* x, void* y, void* stream) {
    try {
        if (!s) return set_error(SELSCAN_ERR_INVALID_ARG, "shape is NULL");
        if (s->n < 1) return set_error(SELSCAN_ERR_INVALID_ARG, "n must be >= 1");
        if (!is_dtype(s->dtype)) return set_error(SELSCAN_ERR_UNSUPPORTED, "dtype must be SELSCAN_F32 or SELSCAN_BF16");
        if (!is_probability(s->p)) return set_error(SELSCAN_ERR_INVALID_ARG, "p must be in [0, 1]");
        if (mul_checked({s->n, 4}) < 0) return set_error(SELSCAN_ERR_INVALID_ARG, "n overflows 64-bit byte counts");
        if (s->n >> 45) return set_error(SELSCAN_ERR_UNSUPPORTED, "too many elements for one launch");
        if (!x || !y) return set_error(SELSCAN_ERR_INVALID_ARG, "x and y must be non-NULL");
        selscan_status_t st = device_check();
        if (st != SELSCAN_OK) return st;
        selscan::DropArgs a{};
        a.x = x; a.y = y; a.n = s->n; a.seed = s->seed; a.offset = s->offset;
        a.keep_from = keep_from(s->p); a.keep_scale = keep_scale(s->p);
        a.vec = aligned16(x) && aligned16(y);
        return launched(selscan::launch_dropout(a, s->dtype == SELSCAN_BF16, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

selscan_status_t selscan_layer_norm_fwd(const selscan_norm_shape_t* s, const void* x, const void* residual,
                                        const float* weight, const float* bias, void* y, void* residual_out,
                                        float* mean, float* rstd, void* stream) {
    try {
        selscan_status_t st = check_norm(s);
        if (st != SELSCAN_OK) return st;
        if (!x || !y) return set_error(SELSCAN_ERR_INVALID_ARG, "x and y must be non-NULL");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        selscan::NormArgs a{};
        fill(a, s);
        a.x = x; a.res = residual; a.weight = weight; a.bias = bias;
        a.y = y; a.res_out = residual_out; a.mean = mean; a.rstd = rstd;
        a.vec = s->dim % 8 == 0 && aligned16(x) && aligned16(residual) && aligned16(y) && aligned16(residual_out) &&
                aligned16(weight) && aligned16(bias);
        return launched(selscan::launch_norm_fwd(a, s->in_dtype == SELSCAN_BF16, s->res_dtype == SELSCAN_BF16,
                                                 s->out_dtype == SELSCAN_BF16, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

size_t selscan_layer_norm_bwd_workspace_bytes(const selscan_norm_shape_t* s) {
    if (check_norm(s) != SELSCAN_OK) return 0;
    return norm_bwd_bytes(s);
}

selscan_status_t selscan_layer_norm_bwd(const selscan_norm_shape_t* s, const void* dy, const void* sum,
                                        const float* weight, const float* mean, const float* rstd,
                                        const void* dresidual_out, void* dx, void* dresidual, float* dweight,
                                        float* dbias, void* stream) {
    try {
        selscan_status_t st = check_norm(s);
        if (st != SELSCAN_OK) return st;
        if (!dy || !sum || !mean || !rstd)
            return set_error(SELSCAN_ERR_INVALID_ARG, "dy, s, mean and rstd must be non-NULL");
        if (!dx && !dresidual && !dweight && !dbias)
            return set_error(SELSCAN_ERR_INVALID_ARG, "one of dx, dresidual, dweight and dbias must be non-NULL");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
        Scratch ws;
        st = ws.get(s->workspace, s->workspace_bytes, dweight || dbias ? norm_bwd_bytes(s) : 0, hs);
        if (st != SELSCAN_OK) return st;
        selscan::NormArgs a{};
        fill(a, s);
        a.x = dy; a.res = sum; a.weight = weight; a.mean_in = mean; a.rstd_in = rstd; a.dres_in = dresidual_out;
        a.y = dx; a.res_out = dresidual; a.dweight = dweight; a.dbias = dbias;
        a.part = static_cast<float*>(ws.ptr);
        a.blocks = selscan::norm_bwd_blocks(s->rows, s->dim);
        a.vec = s->dim % 8 == 0 && aligned16(dy) && aligned16(sum) && aligned16(dresidual_out) && aligned16(dx) &&
                aligned16(dresidual) && aligned16(weight);
        const hipError_t e = selscan::launch_norm_bwd(a, s->in_dtype == SELSCAN_BF16, s->res_dtype == SELSCAN_BF16,
                                                      s->out_dtype == SELSCAN_BF16, hs);
        ws.release();
        return launched(e);
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

}  // extern "C"
