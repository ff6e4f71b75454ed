// rms.cpp -- host side of the RMS norm: argument checks and workspace.
#include <hip/hip_runtime.h>

#include <string>

#include "host.hpp"
#include "kernels.hpp"
#include "selscan.h"

using namespace selscan::host;
using selscan::set_error;

namespace {

bool is_dtype(int32_t d) { return d == SELSCAN_F32 || d == SELSCAN_BF16; }

selscan_status_t check(const selscan_rms_shape_t* s, bool grad) {
    if (!s) return set_error(SELSCAN_ERR_INVALID_ARG, "shape is NULL");
    if (s->rows < 1 || s->dim < 1 || s->groups < 1) return set_error(SELSCAN_ERR_INVALID_ARG, "rows, dim and groups must be >= 1");
    if (s->dim % s->groups != 0) return set_error(SELSCAN_ERR_INVALID_ARG, "dim must be a multiple of groups");
    if (!is_dtype(s->in_dtype) || !is_dtype(s->res_dtype) || !(is_dtype(s->out_dtype) || (!grad && s->out_dtype == SELSCAN_E4M3)))
        return set_error(SELSCAN_ERR_UNSUPPORTED, "dtypes must be SELSCAN_F32 or SELSCAN_BF16 (a forward's y: or SELSCAN_E4M3)");
    const int64_t k = s->scale_block;
    if (k != 0 && k != 32 && k != 64 && k != 128 && k != 256 && k != 512)
        return set_error(SELSCAN_ERR_UNSUPPORTED, "scale_block must be 0, 32, 64, 128, 256 or 512");
    if (!(s->eps >= 0.0f)) return set_error(SELSCAN_ERR_INVALID_ARG, "eps must be >= 0");
    if (s->gate_row < 0) return set_error(SELSCAN_ERR_INVALID_ARG, "gate_row must be >= 0");
    if (mul_checked({s->rows, s->dim, 4}) < 0 || mul_checked({s->rows, s->gate_row, 4}) < 0)
        return set_error(SELSCAN_ERR_INVALID_ARG, "tensor sizes overflow 64-bit byte counts");
    if (s->rows > 0x7fffffff || s->dim > 0x7ffffff || s->groups > 65535)
        return set_error(SELSCAN_ERR_UNSUPPORTED, "the RMS norm supports rows < 2^31, dim < 2^27 and groups < 2^16");
    if (s->rows * s->groups > (int64_t)1 << 35) return set_error(SELSCAN_ERR_UNSUPPORTED, "too many groups for one launch");
    return SELSCAN_OK;
}

int64_t bytes_of(int32_t dtype) { return dtype == SELSCAN_F32 ? 4 : dtype == SELSCAN_BF16 ? 2 : 1; }

// Whether `rows` rows of dim elements at p (dense) overlap those at q (`row`
// elements apart) other than element by element: the kernels read an element
// before they write in its place, and no others.
struct Tensor {
    const void* p;
    int32_t dtype;
    int64_t row;
};
bool in_place(const selscan_rms_shape_t* s, const Tensor& out, const Tensor& in) {
    return out.p == in.p && out.dtype == in.dtype && (in.row == s->dim || s->rows == 1);
}
bool clash(const selscan_rms_shape_t* s, const Tensor& out, const Tensor& in, bool may_be = true) {
    const int64_t eo = bytes_of(out.dtype), ei = bytes_of(in.dtype);
    return out.p && in.p && !(may_be && in_place(s, out, in)) &&
           overlap(out.p, s->rows * s->dim * eo, in.p, s->dim * ei, s->rows, in.row * ei);
}

void fill(selscan::RmsArgs& a, const selscan_rms_shape_t* s) {
    a.rows = s->rows; a.dim = s->dim; a.groups = s->groups; a.gate_row = s->gate_row;
    a.width = s->dim / s->groups;
    a.block = s->scale_block;
    a.row_blocks = a.block ? (a.width + a.block - 1) / a.block : 1;
    a.eps = s->eps;
    a.inv_width = (float)(1.0 / (double)a.width);
}

size_t part_bytes(const selscan_rms_shape_t* s) { return align256(selscan::rms_bwd_part_bytes(s->rows, s->dim, s->groups)); }

selscan_status_t launched(hipError_t e) {
    if (e != hipSuccess)
        return set_error(SELSCAN_ERR_LAUNCH, std::string("kernel launch failed: ") + hipGetErrorString(e));
    return set_error(SELSCAN_OK, "");
}

}  // namespace

extern "C" {

selscan_status_t selscan_rms_norm_fwd(const selscan_rms_shape_t* s, const void* x, const void* residual, const void* gate,
                                      const float* weight, void* y, void* residual_out, float* rstd, float* scale,
                                      void* stream) {
    try {
        selscan_status_t st = check(s, false);
        if (st != SELSCAN_OK) return st;
        if (!x || !y) return set_error(SELSCAN_ERR_INVALID_ARG, "x and y must be non-NULL");
        if (gate && (residual || residual_out))
            return set_error(SELSCAN_ERR_UNSUPPORTED, "a gate takes neither residual nor residual_out");
        if (s->out_dtype == SELSCAN_E4M3 && !scale)
            return set_error(SELSCAN_ERR_INVALID_ARG, "scale must be non-NULL where y is in 8 bits");
        const Tensor outs[] = {{y, s->out_dtype, s->dim}, {residual_out, s->res_dtype, s->dim}};
        const Tensor ins[] = {{x, s->in_dtype, s->dim}, {residual, s->res_dtype, s->dim}, {gate, s->in_dtype, s->gate_row}};
        bool bad = clash(s, outs[0], outs[1], false);
        for (const Tensor& o : outs)
            for (const Tensor& i : ins) bad = bad || clash(s, o, i);
        if (bad)
            return set_error(SELSCAN_ERR_INVALID_ARG, "y and residual_out must not alias each other, nor inputs but in the place and type of one");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        selscan::RmsArgs a{};
        fill(a, s);
        a.x = x; a.res = residual; a.gate = gate; a.weight = weight; a.y = y; a.res_out = residual_out;
        a.rstd = rstd; a.scale = scale;
        return launched(selscan::launch_rms_fwd(a, s->in_dtype == SELSCAN_BF16, s->res_dtype == SELSCAN_BF16, s->out_dtype,
                                                reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

size_t selscan_rms_norm_bwd_workspace_bytes(const selscan_rms_shape_t* s) {
    if (check(s, true) != SELSCAN_OK) return 0;
    return part_bytes(s);
}

selscan_status_t selscan_rms_norm_bwd(const selscan_rms_shape_t* s, const void* dy, const void* sum, const void* gate,
                                      const float* weight, const float* rstd, const void* dresidual_out, void* dx,
                                      void* dresidual, void* dgate, float* dweight, void* stream) {
    try {
        selscan_status_t st = check(s, true);
        if (st != SELSCAN_OK) return st;
        if (!dy || !sum || !rstd) return set_error(SELSCAN_ERR_INVALID_ARG, "dy, s and rstd must be non-NULL");
        if (!dx && !dresidual && !dgate && !dweight)
            return set_error(SELSCAN_ERR_INVALID_ARG, "one of dx, dresidual, dgate and dweight must be non-NULL");
        if (gate && (dresidual_out || dresidual))
            return set_error(SELSCAN_ERR_UNSUPPORTED, "a gate takes neither dresidual_out nor dresidual");
        if (gate && s->res_dtype != s->in_dtype)
            return set_error(SELSCAN_ERR_UNSUPPORTED, "with a gate, s is x: res_dtype must be in_dtype");
        if (!gate && dgate) return set_error(SELSCAN_ERR_INVALID_ARG, "dgate needs gate");
        const Tensor outs[] = {{dx, s->in_dtype, s->dim}, {dresidual, s->res_dtype, s->dim}, {dgate, s->in_dtype, s->dim}};
        const Tensor ins[] = {{dy, s->out_dtype, s->dim}, {sum, s->res_dtype, s->dim}, {gate, s->in_dtype, s->gate_row}};
        // long groups: dweight is made from dy, s and gate when the gradients are there
        const bool again = dweight && selscan::rms_reads_again(s->dim / s->groups);
        bool bad = clash(s, outs[0], outs[1], false) || clash(s, outs[0], outs[2], false);
        for (const Tensor& o : outs) {
            bad = bad || clash(s, o, {dresidual_out, s->res_dtype, s->dim});
            for (const Tensor& i : ins) bad = bad || clash(s, o, i, !again);
        }
        if (bad)
            return set_error(SELSCAN_ERR_INVALID_ARG, "gradients must not alias each other, nor inputs but in the place and type of one "
                                                      "(dy, s and gate: not with dweight of groups past 8192)");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
        Scratch ws;
        st = ws.get(s->workspace, s->workspace_bytes, dweight ? part_bytes(s) : 0, hs);
        if (st != SELSCAN_OK) return st;
        selscan::RmsArgs a{};
        fill(a, s);
        a.x = dy; a.res = sum; a.gate = gate; a.weight = weight; a.rstd_in = rstd; a.dres_in = dresidual_out;
        a.y = dx; a.res_out = dresidual; a.dgate = dgate; a.dweight = dweight;
        a.part = static_cast<float*>(ws.ptr);
        a.blocks = selscan::rms_bwd_blocks(a.rows, a.width);
        const hipError_t e = selscan::launch_rms_bwd(a, s->in_dtype == SELSCAN_BF16, s->res_dtype == SELSCAN_BF16,
                                                     s->out_dtype == SELSCAN_BF16, hs);
        ws.release();
        return launched(e);
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

}  // extern "C"
