// mixer.cpp -- host side of the short convolution and of the Mamba-2 mixer
// with it in front: argument checks, plans and workspace.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "host.hpp"
#include "kernels.hpp"
#include "selscan.h"

using namespace selscan::host;
using selscan::set_error;

namespace {

constexpr int64_t kMostGroups = (int64_t)1 << 35;   // workgroups of a launch over two grid dimensions

// What the sums of partial rows take in one launch: (width + 1) dim columns at
// 16 threads each, fewer than 2^32, and 65535 times 1024 rows.
constexpr int64_t kMostSumCols = (int64_t)1 << 24, kMostSumRows = (int64_t)1 << 25;

bool is_dtype(int32_t d) { return d == SELSCAN_F32 || d == SELSCAN_BF16; }
int64_t bytes_of(int32_t dtype) { return dtype == SELSCAN_F32 ? 4 : 2; }

selscan_status_t check_width(int64_t width) {
    if (width < 1) return set_error(SELSCAN_ERR_INVALID_ARG, "width must be >= 1");
    if (width < 2 || width > 4) return set_error(SELSCAN_ERR_UNSUPPORTED, "the short convolution supports width 2, 3, 4");
    return SELSCAN_OK;
}

// Rows of `dim` elements, strided: the byte offset of the last one fits.
bool strides_fit(int64_t batch, int64_t b_stride, int64_t rows, int64_t stride, int64_t dim) {
    if (b_stride < 0 || stride < 0) return false;
    const int64_t x = mul_checked({batch, b_stride}), y = mul_checked({rows, stride});
    return x >= 0 && y >= 0 && x < INT64_MAX / 16 && y < INT64_MAX / 16 && dim < INT64_MAX / 16;
}

enum Use { kSequence, kGrad, kToken };

void fill(selscan::ShortConvArgs& a, const selscan_short_conv_shape_t* s, Use use) {
    a.batch = s->batch; a.L = use == kToken ? 1 : s->seqlen; a.C = s->dim; a.K = (int)s->width;
    a.x_row = s->x_row; a.x_batch = s->x_batch;
    a.begin[0] = 0;
    a.begin[1] = use == kToken ? s->dim : s->split[0];
    a.begin[2] = use == kToken ? s->dim : s->split[0] + s->split[1];
    selscan::short_conv_plan(a, use == kGrad);
}

selscan_status_t check_conv(const selscan_short_conv_shape_t* s, Use use) {
    if (!s) return set_error(SELSCAN_ERR_INVALID_ARG, "shape is NULL");
    const int64_t L = use == kToken ? 1 : s->seqlen;
    if (s->batch < 1 || L < 1 || s->dim < 1) return set_error(SELSCAN_ERR_INVALID_ARG, "batch, seqlen and dim must be >= 1");
    selscan_status_t st = check_width(s->width);
    if (st != SELSCAN_OK) return st;
    if (!is_dtype(s->in_dtype) || !is_dtype(s->out_dtype))
        return set_error(SELSCAN_ERR_UNSUPPORTED, "dtypes must be SELSCAN_F32 or SELSCAN_BF16");
    if (mul_checked({s->batch, L, s->dim, 4}) < 0 || mul_checked({s->batch, s->dim, 16}) < 0)
        return set_error(SELSCAN_ERR_INVALID_ARG, "tensor sizes overflow 64-bit byte counts");
    if (!strides_fit(s->batch, s->x_batch, L, use == kToken ? 0 : s->x_row, s->dim))
        return set_error(SELSCAN_ERR_INVALID_ARG, "x_row and x_batch must be >= 0 and their offsets fit 64 bits");
    if (use != kToken) {
        if (s->split[0] < 1 || s->split[1] < 0 || s->split[2] < 0 || s->split[0] > s->dim || s->split[1] > s->dim ||
            s->split[2] > s->dim || s->split[0] + s->split[1] + s->split[2] != s->dim)
            return set_error(SELSCAN_ERR_INVALID_ARG, "split must be channels of the outputs, dim in all, the first >= 1");
        selscan::ShortConvArgs a{};
        fill(a, s, use);
        const int64_t blocks = mul_checked({a.batch, a.run_blocks, a.col_blocks});
        if (blocks < 0 || blocks > kMostGroups ||
            (use == kGrad && mul_checked({a.batch, a.run_blocks, s->width + 1, s->dim, 8}) < 0))
            return set_error(SELSCAN_ERR_UNSUPPORTED, "too many elements for one launch");
        if (use == kGrad && (s->dim > kMostSumCols || a.batch * a.run_blocks > kMostSumRows))
            return set_error(SELSCAN_ERR_UNSUPPORTED, "the short convolution's gradients support dim <= 2^24 and up to 2^25 blocks of rows");
    }
    if (s->dim > (int64_t)1 << 32 || s->batch > (int64_t)1 << 31 ||
        mul_checked({s->batch, s->dim}) / 256 > kMostGroups)
        return set_error(SELSCAN_ERR_UNSUPPORTED, "the short convolution supports dim <= 2^32 and batch <= 2^31");
    return SELSCAN_OK;
}

// Dense tensors by their bytes (p NULL: none), of which an output must overlap
// neither another nor an input.
struct Span {
    const void* p;
    int64_t bytes;
};
bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        if (!o->p) continue;
        for (const Span* i = o + 1; i != outs.end(); ++i)
            if (i->p && overlap(o->p, o->bytes, i->p, i->bytes)) return false;
        for (const Span& i : ins)
            if (i.p && overlap(o->p, o->bytes, i.p, i.bytes)) return false;
    }
    return true;
}
// The outputs and rows that a projection left, [batch, rows] of them.
bool apart(std::initializer_list<Span> outs, const void* q, int64_t bytes, int64_t rows, int64_t stride, int64_t batch, int64_t b_stride) {
    for (const Span& o : outs)
        if (o.p && overlap(o.p, o.bytes, q, bytes, rows, stride, batch, b_stride)) return false;
    return true;
}

size_t conv_part_bytes(const selscan::ShortConvArgs& a) {
    return align256((size_t)selscan::column_sums_rows(a.batch * a.run_blocks) * (size_t)((a.K + 1) * a.C) * 4);
}

selscan_status_t launched(hipError_t e) {
    if (e != hipSuccess)
        return set_error(SELSCAN_ERR_LAUNCH, std::string("kernel launch failed: ") + hipGetErrorString(e));
    return set_error(SELSCAN_OK, "");
}

selscan_status_t check_mixer(const selscan_m2_conv_shape_t* s, bool token) {
    if (!s) return set_error(SELSCAN_ERR_INVALID_ARG, "shape is NULL");
    const int64_t L = token ? 1 : s->seqlen;
    if (s->batch < 1 || L < 1 || s->nheads < 1 || s->headdim < 1 || s->ngroups < 1 || s->dstate < 1)
        return set_error(SELSCAN_ERR_INVALID_ARG, "batch, seqlen, nheads, headdim, ngroups, dstate must be >= 1");
    if (s->nheads % s->ngroups != 0) return set_error(SELSCAN_ERR_INVALID_ARG, "nheads must be a multiple of ngroups");
    if (s->dstate != 16 && s->dstate != 32 && s->dstate != 64 && s->dstate != 128)
        return set_error(SELSCAN_ERR_UNSUPPORTED, "the Mamba-2 mixer supports dstate 16, 32, 64, 128");
    selscan_status_t st = check_width(s->width);
    if (st != SELSCAN_OK) return st;
    if (!is_dtype(s->in_dtype) || !is_dtype(s->out_dtype))
        return set_error(SELSCAN_ERR_UNSUPPORTED, "dtypes must be SELSCAN_F32 or SELSCAN_BF16");
    const int64_t hp = mul_checked({s->nheads, s->headdim}), gn = mul_checked({s->ngroups, s->dstate});
    if (hp < 0 || gn < 0 || hp > INT64_MAX / 4 || gn > INT64_MAX / 8 || mul_checked({s->batch, L, hp + 2 * gn, 4}) < 0 ||
        mul_checked({s->batch, hp, s->dstate, 4}) < 0 || mul_checked({s->batch, hp + 2 * gn, 16}) < 0)
        return set_error(SELSCAN_ERR_INVALID_ARG, "tensor sizes overflow 64-bit byte counts");
    if (!strides_fit(s->batch, s->xbc_batch, L, token ? 0 : s->xbc_row, hp + 2 * gn) ||
        !strides_fit(s->batch, s->dt_batch, L, token ? 0 : s->dt_row, s->nheads))
        return set_error(SELSCAN_ERR_INVALID_ARG, "strides must be >= 0 and their offsets fit 64 bits");
    if (hp + 2 * gn > (int64_t)1 << 22 || mul_checked({s->batch, s->nheads, (s->headdim + 15) / 16}) > kMostGroups ||
        s->batch > (int64_t)1 << 31)
        return set_error(SELSCAN_ERR_UNSUPPORTED, "the Mamba-2 mixer supports up to 2^22 channels of xbc, and rows of states for one launch");
    if (!token) {
        // a record of a chunk's B and C is at most 2^17 bytes, and a GPU's
        // compute units ask for fewer than 2^12 segments of a sequence
        const int64_t chunks = (L + 63) / 64;
        const int64_t recs = mul_checked({s->batch, chunks, s->ngroups, (int64_t)1 << 17});
        if (recs < 0 || recs >> 17 > kMostGroups || mul_checked({s->batch, hp, s->dstate, 4, 4096}) < 0 ||
            mul_checked({s->batch, hp, s->dstate}) / 256 > kMostGroups)
            return set_error(SELSCAN_ERR_UNSUPPORTED, "too many chunks or states for one launch");
    }
    return SELSCAN_OK;
}

void fill(selscan::M2ConvArgs& a, const selscan_m2_conv_shape_t* s, bool token) {
    a.batch = s->batch; a.L = token ? 1 : s->seqlen; a.H = s->nheads; a.P = s->headdim; a.G = s->ngroups; a.N = s->dstate;
    a.dt_row = s->dt_row; a.dt_batch = s->dt_batch;
    a.conv.batch = a.batch; a.conv.L = a.L; a.conv.C = a.H * a.P + 2 * a.G * a.N; a.conv.K = (int)s->width;
    a.conv.x_row = s->xbc_row; a.conv.x_batch = s->xbc_batch;
    a.conv.silu = 1;
    a.conv.begin[0] = 0;
    a.conv.begin[1] = token ? a.conv.C : a.H * a.P;
    a.conv.begin[2] = token ? a.conv.C : a.H * a.P + a.G * a.N;
    selscan::short_conv_plan(a.conv, false);
}

// Short sequences are walked token by token, in a time that goes with their
// length; in chunks it hardly moves within one.  us, token by token / in chunks,
// bf16, heads of 64 x 128, from a state of zero and from h0 (whose states are
// read too):
//              32 heads       256 heads      512 heads      2048 heads     4096 heads
//   L =  4     8.5 / 30.0    11.1 / 31.0    14.7 / 32.3    32.7 /  55.8    55.2 /  93.7
//     h0       8.9 / 33.4    13.7 / 34.3    21.9 / 37.2    58.6 /  64.7   111.9 / 117.3
//   L =  8    10.6 / 29.9    13.4 / 30.9    20.0 / 32.1    51.2 /  55.8    90.5 /  94.1
//     h0      11.0 / 33.4    16.2 / 34.3    26.9 / 37.3    76.6 /  64.9   150.3 / 118.1
//   L = 16    15.0 / 30.1    18.1 / 31.0    30.1 / 32.2    87.5 /  56.2   160.8 /  94.4
//     h0      15.3 / 33.6    21.0 / 34.5    36.9 / 37.5   112.9 /  65.0   226.6 / 120.9
//   L = 32    22.4 / 30.2    27.8 / 31.3    52.9 / 32.5   159.1 /  56.7   296.4 /  95.4
//     h0      22.8 / 33.8    30.7 / 34.9    59.3 / 37.5   184.8 /  65.5   370.2 / 125.9
// The two meet at 38 tokens (256 heads, 2^21 elements of state), 16 (512), and
// from 2048 heads on, where both go with the states, at 9 from zero and 5 from
// h0, whatever the number.  (fp32's chunks take less up to 512 heads, 24 to 30
// us, and more from there; heads of 64 x 16 as many as 32 meet at 33.)
constexpr int64_t kRecTokens = 32, kRecTokensFull = 7;

// The chunked form's offsets inside 64 tokens and the three before are 32-bit.
bool chunked(const selscan::M2ConvArgs& a) {
    const int64_t fills = std::max<int64_t>(1, a.batch * a.H * a.P * a.N >> 21);
    return a.L > std::max(kRecTokens / fills, kRecTokensFull) && a.conv.x_row < ((int64_t)1 << 30) / (4 * 68);
}

size_t mixer_bytes(const selscan::M2ConvArgs& a, int in_bf16) {
    return chunked(a) ? selscan::m2_chunk_bytes(a, in_bf16) : selscan::m2_rec_bytes(a);
}

}  // namespace

extern "C" {

selscan_status_t selscan_short_conv_fwd(const selscan_short_conv_shape_t* s, const void* x, const float* weight,
                                        const float* bias, int silu, const int32_t* lengths, const void* state, void* y0,
                                        void* y1, void* y2, void* last_state, void* stream) {
    try {
        selscan_status_t st = check_conv(s, kSequence);
        if (st != SELSCAN_OK) return st;
        if (!x || !weight || !y0 || (s->split[1] && !y1) || (s->split[2] && !y2))
            return set_error(SELSCAN_ERR_INVALID_ARG, "x, weight and the outputs of split must be non-NULL");
        if (silu != 0 && silu != 1) return set_error(SELSCAN_ERR_INVALID_ARG, "silu must be 0 or 1");
        const int64_t es = bytes_of(s->in_dtype), n = s->batch * s->seqlen * bytes_of(s->out_dtype);
        const int64_t ns = s->batch * (s->width - 1) * s->dim * es;
        const std::initializer_list<Span> outs = {{y0, n * s->split[0]}, {s->split[1] ? y1 : nullptr, n * s->split[1]},
                                                  {s->split[2] ? y2 : nullptr, n * s->split[2]}, {last_state, ns}};
        if (!apart(outs, {{state, ns}}) || !apart(outs, x, s->dim * es, s->seqlen, s->x_row * es, s->batch, s->x_batch * es))
            return set_error(SELSCAN_ERR_INVALID_ARG, "the outputs and last_state must not alias x, state or each other");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        selscan::ShortConvArgs a{};
        fill(a, s, kSequence);
        a.x = x; a.weight = weight; a.bias = bias; a.silu = silu; a.lengths = lengths; a.state = state;
        a.y[0] = y0; a.y[1] = y1; a.y[2] = y2; a.last = last_state;
        return launched(selscan::launch_short_conv_fwd(a, s->in_dtype == SELSCAN_BF16, s->out_dtype == SELSCAN_BF16,
                                                       reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

size_t selscan_short_conv_bwd_workspace_bytes(const selscan_short_conv_shape_t* s) {
    if (check_conv(s, kGrad) != SELSCAN_OK) return 0;
    selscan::ShortConvArgs a{};
    fill(a, s, kGrad);
    return conv_part_bytes(a);
}

selscan_status_t selscan_short_conv_bwd(const selscan_short_conv_shape_t* s, const void* x, const float* weight,
                                        const float* bias, int silu, const int32_t* lengths, const void* state,
                                        const void* dout0, const void* dout1, const void* dout2, const void* dlast_state,
                                        void* dx, float* dweight, float* dbias, void* dstate, void* stream) {
    try {
        selscan_status_t st = check_conv(s, kGrad);
        if (st != SELSCAN_OK) return st;
        if (!x || !weight || !dx || !dout0 || (s->split[1] && !dout1) || (s->split[2] && !dout2))
            return set_error(SELSCAN_ERR_INVALID_ARG, "x, weight, dx and the gradients of split must be non-NULL");
        if (silu != 0 && silu != 1) return set_error(SELSCAN_ERR_INVALID_ARG, "silu must be 0 or 1");
        const int64_t es = bytes_of(s->in_dtype), n = s->batch * s->seqlen, ny = n * bytes_of(s->out_dtype);
        const int64_t ns = s->batch * (s->width - 1) * s->dim * es;
        const std::initializer_list<Span> outs = {{dx, n * s->dim * es}, {dweight, s->dim * s->width * 4}, {dbias, s->dim * 4}, {dstate, ns}};
        if (!apart(outs, {{dout0, ny * s->split[0]}, {s->split[1] ? dout1 : nullptr, ny * s->split[1]},
                          {s->split[2] ? dout2 : nullptr, ny * s->split[2]}, {state, ns}, {dlast_state, ns}}) ||
            !apart(outs, x, s->dim * es, s->seqlen, s->x_row * es, s->batch, s->x_batch * es))
            return set_error(SELSCAN_ERR_INVALID_ARG, "gradients must not alias inputs or each other");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
        selscan::ShortConvArgs a{};
        fill(a, s, kGrad);
        Scratch ws;
        st = ws.get(s->workspace, s->workspace_bytes, dweight || dbias ? conv_part_bytes(a) : 0, hs);
        if (st != SELSCAN_OK) return st;
        a.x = x; a.weight = weight; a.bias = bias; a.silu = silu; a.lengths = lengths; a.state = state;
        a.dout[0] = dout0; a.dout[1] = dout1; a.dout[2] = dout2; a.dlast = dlast_state;
        a.dx = dx; a.dweight = dweight; a.dbias = dbias; a.dstate = dstate;
        a.part = static_cast<float*>(ws.ptr);
        const hipError_t e = selscan::launch_short_conv_bwd(a, s->in_dtype == SELSCAN_BF16, s->out_dtype == SELSCAN_BF16, hs);
        ws.release();
        return launched(e);
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

selscan_status_t selscan_short_conv_step(const selscan_short_conv_shape_t* s, void* state, const void* x,
                                         const float* weight, const float* bias, int silu, void* y, void* stream) {
    try {
        selscan_status_t st = check_conv(s, kToken);
        if (st != SELSCAN_OK) return st;
        if (!state || !x || !weight || !y)
            return set_error(SELSCAN_ERR_INVALID_ARG, "state, x, weight and y must be non-NULL");
        if (silu != 0 && silu != 1) return set_error(SELSCAN_ERR_INVALID_ARG, "silu must be 0 or 1");
        // (a thread reads its channels of a row before it writes them)
        const int64_t es = bytes_of(s->in_dtype), ny = s->batch * s->dim * bytes_of(s->out_dtype);
        const int64_t ns = s->batch * (s->width - 1) * s->dim * es;
        const bool in_place = y == x && s->in_dtype == s->out_dtype && (s->batch == 1 || s->x_batch == s->dim);
        if ((!in_place && overlap(y, ny, x, s->dim * es, s->batch, s->x_batch * es)) || overlap(y, ny, state, ns) ||
            overlap(state, ns, x, s->dim * es, s->batch, s->x_batch * es))
            return set_error(SELSCAN_ERR_INVALID_ARG, "y must not alias x (but be x, of its type and dense) or state, nor state x");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        selscan::ShortConvArgs a{};
        fill(a, s, kToken);
        a.x = x; a.weight = weight; a.bias = bias; a.silu = silu; a.last = state; a.y[0] = y;
        return launched(selscan::launch_short_conv_step(a, s->in_dtype == SELSCAN_BF16, s->out_dtype == SELSCAN_BF16,
                                                        reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

size_t selscan_mamba2_conv_workspace_bytes(const selscan_m2_conv_shape_t* s) {
    if (check_mixer(s, false) != SELSCAN_OK) return 0;
    selscan::M2ConvArgs a{};
    fill(a, s, false);
    return mixer_bytes(a, s->in_dtype == SELSCAN_BF16);
}

selscan_status_t selscan_mamba2_conv_fwd(const selscan_m2_conv_shape_t* s, const void* xbc, const void* dt,
                                         const float* conv_weight, const float* conv_bias, const float* A, const float* D,
                                         const float* dt_bias, const int32_t* lengths, const float* h0,
                                         const void* conv_state, void* y, float* last_state, void* last_conv_state,
                                         void* stream) {
    try {
        selscan_status_t st = check_mixer(s, false);
        if (st != SELSCAN_OK) return st;
        if (!xbc || !dt || !conv_weight || !A || !y)
            return set_error(SELSCAN_ERR_INVALID_ARG, "xbc, dt, conv_weight, A and y must be non-NULL");
        const int64_t hp = s->nheads * s->headdim, C = hp + 2 * s->ngroups * s->dstate, es = bytes_of(s->in_dtype);
        const int64_t ns = s->batch * hp * s->dstate * 4, nc = s->batch * (s->width - 1) * C * es;
        const std::initializer_list<Span> outs = {{y, s->batch * s->seqlen * hp * bytes_of(s->out_dtype)}, {last_state, ns}, {last_conv_state, nc}};
        if (!apart(outs, {{h0, ns}, {conv_state, nc}}) ||
            !apart(outs, xbc, C * es, s->seqlen, s->xbc_row * es, s->batch, s->xbc_batch * es) ||
            !apart(outs, dt, s->nheads * es, s->seqlen, s->dt_row * es, s->batch, s->dt_batch * es))
            return set_error(SELSCAN_ERR_INVALID_ARG, "y, last_state and last_conv_state must not alias inputs or each other");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
        selscan::M2ConvArgs a{};
        fill(a, s, false);
        Scratch ws;
        st = ws.get(s->workspace, s->workspace_bytes, mixer_bytes(a, s->in_dtype == SELSCAN_BF16), hs);
        if (st != SELSCAN_OK) return st;
        a.conv.x = xbc; a.conv.weight = conv_weight; a.conv.bias = conv_bias; a.conv.lengths = lengths;
        a.conv.state = conv_state; a.conv.last = last_conv_state;
        a.dt = dt; a.A = A; a.D = D; a.dt_bias = dt_bias; a.h0 = h0; a.y = y; a.last = last_state;
        const auto launch = chunked(a) ? &selscan::launch_m2_chunk : &selscan::launch_m2_rec;
        const hipError_t e = launch(a, s->in_dtype == SELSCAN_BF16, s->out_dtype == SELSCAN_BF16, ws.ptr, hs);
        ws.release();
        return launched(e);
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

selscan_status_t selscan_mamba2_conv_step(const selscan_m2_conv_shape_t* s, float* state, void* conv_state, const void* xbc,
                                          const void* dt, const float* conv_weight, const float* conv_bias, const float* A,
                                          const float* D, const float* dt_bias, void* y, void* stream) {
    try {
        selscan_status_t st = check_mixer(s, true);
        if (st != SELSCAN_OK) return st;
        if (!state || !conv_state || !xbc || !dt || !conv_weight || !A || !y)
            return set_error(SELSCAN_ERR_INVALID_ARG, "state, conv_state, xbc, dt, conv_weight, A and y must be non-NULL");
        if (!aligned16(state)) return set_error(SELSCAN_ERR_INVALID_ARG, "state must be 16-byte aligned");
        // y is written while other workgroups read dt and the channels of B and C,
        // and a launch behind that reads all of xbc
        const int64_t hp = s->nheads * s->headdim, C = hp + 2 * s->ngroups * s->dstate;
        const int64_t es = bytes_of(s->in_dtype), ny = s->batch * hp * bytes_of(s->out_dtype);
        const int64_t ns = s->batch * hp * s->dstate * 4, nc = s->batch * (s->width - 1) * C * es;
        const auto inputs = [&](const void* p, int64_t n) {
            return overlap(p, n, xbc, C * es, s->batch, s->xbc_batch * es) ||
                   overlap(p, n, dt, s->nheads * es, s->batch, s->dt_batch * es);
        };
        if (inputs(y, ny) || inputs(state, ns) || inputs(conv_state, nc) || overlap(y, ny, state, ns) ||
            overlap(y, ny, conv_state, nc) || overlap(state, ns, conv_state, nc))
            return set_error(SELSCAN_ERR_INVALID_ARG, "y, state and conv_state must not alias xbc, dt or each other");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        selscan::M2ConvArgs a{};
        fill(a, s, true);
        a.conv.x = xbc; a.conv.weight = conv_weight; a.conv.bias = conv_bias;
        a.conv.state = conv_state; a.conv.last = conv_state;
        a.dt = dt; a.A = A; a.D = D; a.dt_bias = dt_bias; a.last = state; a.y = y;
        return launched(selscan::launch_m2_conv_step(a, s->in_dtype == SELSCAN_BF16, s->out_dtype == SELSCAN_BF16,
                                                     reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

}  // extern "C"
