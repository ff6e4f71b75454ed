// delta.cpp -- host side of the gated delta rule: argument checks, plans and
// workspace behind the entry points declared in selscan.h.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <string>

#include "host.hpp"
#include "kernels.hpp"
#include "selscan.h"

using namespace selscan::host;
using selscan::set_error;

namespace {

selscan_status_t check_shape(const selscan_m2_shape_t* s) {
    if (!s) return set_error(SELSCAN_ERR_INVALID_ARG, "shape is NULL");
    if (s->batch < 1 || s->seqlen < 1 || s->nheads < 1 || s->headdim < 1 || s->ngroups < 1 || s->dstate < 1)
        return set_error(SELSCAN_ERR_INVALID_ARG, "batch, seqlen, nheads, headdim, ngroups, dstate must be >= 1");
    if (s->nheads % s->ngroups != 0)
        return set_error(SELSCAN_ERR_INVALID_ARG, "nheads must be a multiple of ngroups");
    if (s->dstate > 128) return set_error(SELSCAN_ERR_UNSUPPORTED, "the gated delta rule supports dstate <= 128");
    if ((s->in_dtype != SELSCAN_F32 && s->in_dtype != SELSCAN_BF16) ||
        (s->out_dtype != SELSCAN_F32 && s->out_dtype != SELSCAN_BF16))
        return set_error(SELSCAN_ERR_UNSUPPORTED, "dtypes must be SELSCAN_F32 or SELSCAN_BF16");
    if (mul_checked({s->batch, s->seqlen, s->nheads, s->headdim, 4}) < 0 ||
        mul_checked({s->batch, s->seqlen, s->ngroups, s->dstate, 4}) < 0 ||
        mul_checked({s->batch, s->nheads, s->headdim, s->dstate, 4}) < 0)
        return set_error(SELSCAN_ERR_INVALID_ARG, "tensor sizes overflow 64-bit byte counts");
    // the chunked form's offsets inside 64 tokens are 32-bit
    if (s->nheads * s->headdim > (int64_t(1) << 22) || s->ngroups > (int64_t(1) << 15))
        return set_error(SELSCAN_ERR_UNSUPPORTED, "the gated delta rule supports nheads headdim <= 2^22 and ngroups <= 2^15");
    // a launch has fewer than 2^32 threads: 512 to 16 rows of a head's state, 64
    // to a chunk (whose limit is lower: 2^24 chunks' records are 512 GB)
    const int64_t heads = (s->batch * s->nheads + 7) / 8 * 8;
    if (heads * ((s->headdim + 15) / 16) >= 1 << 23 || mul_checked({heads, selscan::delta_chunks(s->seqlen)}) >= 1 << 24)
        return set_error(SELSCAN_ERR_UNSUPPORTED, "too many (batch, head, channel) rows or chunks for one launch");
    return SELSCAN_OK;
}

bool vec4(const selscan_m2_shape_t* s, const void* q, const void* k) {
    const uintptr_t m = s->in_dtype == SELSCAN_BF16 ? 7 : 15;
    return s->dstate % 4 == 0 && (reinterpret_cast<uintptr_t>(q) & m) == 0 && (reinterpret_cast<uintptr_t>(k) & m) == 0;
}

// Sequences longer than this take the chunked form, whose time hardly moves
// within a chunk, where the token-by-token form's is proportional to the
// length.  us, token by token / chunked, at bf16, 128 x 128 states:
//              16 heads     128 heads      1024 heads
//   L =  8    7.5 / 14.3   11.5 / 25.0    58.1 / 115.3
//   L = 16   12.1 / 14.6   17.8 / 25.2    96.3 / 115.0
//   L = 24   16.9 / 15.0   23.6 / 25.5   135.3 / 115.1
//   L = 32   21.4 / 15.5   28.9 / 25.9   175.3 / 116.8
//   L = 64   39.7 / 16.6   71.1 / 27.4   333.1 / 123.2
constexpr int64_t kRecTokens = 16;

// Padded copies of q and k, which rows that are not made of 16-byte pieces take.
size_t pad_bytes(const selscan_m2_shape_t* s) {
    return align256((size_t)(s->batch * s->seqlen * s->ngroups) * 2 * (s->dstate <= 64 ? 64 : 128) *
                    (s->in_dtype == SELSCAN_BF16 ? 2 : 4));
}

size_t record_bytes(const selscan_m2_shape_t* s) {
    return align256((size_t)(s->batch * s->nheads * selscan::delta_chunks(s->seqlen)) * selscan::delta_record_bytes(false));
}

size_t fwd_bytes(const selscan_m2_shape_t* s) {
    if (s->seqlen <= kRecTokens) return 0;
    return record_bytes(s) + (s->dstate % 8 ? pad_bytes(s) : 0);
}

// The copies' place: after the call's other workspace when N asks for them
// whatever the addresses, else (q or k off a 16-byte boundary) their own.
selscan_status_t pad_rows(selscan::DeltaArgs& a, const selscan_m2_shape_t* s, char* after, Scratch& own, hipStream_t hs) {
    a.NL = a.N;
    a.qk_row = a.N;
    if (a.N % 8 == 0) {
        if (aligned16(a.q) && aligned16(a.k)) return SELSCAN_OK;
        const selscan_status_t st = own.get(nullptr, 0, pad_bytes(s), hs);
        if (st != SELSCAN_OK) return st;
        after = static_cast<char*>(own.ptr);
    }
    const hipError_t e = selscan::launch_delta_pad(a, s->in_dtype == SELSCAN_BF16, after, hs);
    if (e != hipSuccess)
        return set_error(SELSCAN_ERR_LAUNCH, std::string("kernel launch failed: ") + hipGetErrorString(e));
    return SELSCAN_OK;
}

selscan_status_t check_bwd_shape(const selscan_m2_shape_t* s) {
    selscan_status_t st = check_shape(s);
    if (st != SELSCAN_OK) return st;
    if (mul_checked({s->batch, s->nheads, selscan::delta_chunks(s->seqlen), (s->headdim + 31) / 32 * 32, 128, 16}) < 0 ||
        mul_checked({s->batch, s->seqlen, s->nheads, s->dstate, 16}) < 0)
        return set_error(SELSCAN_ERR_INVALID_ARG, "workspace size overflows 64-bit byte counts");
    // 512 threads to 16 of the rows of a head's state, which are padded to a
    // multiple of 32 here, and 512 to a chunk
    const int64_t heads = (s->batch * s->nheads + 7) / 8 * 8;
    if (heads * ((s->headdim + 31) / 32 * 2) >= 1 << 23 || s->batch * s->nheads * selscan::delta_chunks(s->seqlen) >= 1 << 23)
        return set_error(SELSCAN_ERR_UNSUPPORTED, "too many (batch, head, channel) rows or chunks for one launch");
    return SELSCAN_OK;
}

size_t bwd_main_bytes(const selscan_m2_shape_t* s) {
    return selscan::delta_bwd_bytes(s->batch, s->seqlen, s->nheads, s->ngroups, s->headdim, s->dstate);
}

size_t bwd_bytes(const selscan_m2_shape_t* s) { return bwd_main_bytes(s) + (s->dstate % 8 ? pad_bytes(s) : 0); }

selscan_status_t launched(hipError_t e) {
    if (e != hipSuccess)
        return set_error(SELSCAN_ERR_LAUNCH, std::string("kernel launch failed: ") + hipGetErrorString(e));
    return set_error(SELSCAN_OK, "");
}

}  // namespace

extern "C" {

size_t selscan_delta_workspace_bytes(const selscan_m2_shape_t* s) {
    if (check_shape(s) != SELSCAN_OK) return 0;
    return fwd_bytes(s);
}

selscan_status_t selscan_delta_fwd(const selscan_m2_shape_t* s, const void* q, const void* k, const void* v,
                                   const float* g, const float* beta, float scale, const int32_t* lengths,
                                   const float* h0, void* y, float* last_state, void* stream) {
    try {
        selscan_status_t st = check_shape(s);
        if (st != SELSCAN_OK) return st;
        if (!q || !k || !v || !g || !beta || !y)
            return set_error(SELSCAN_ERR_INVALID_ARG, "q, k, v, g, beta and y must be non-NULL");
        if (h0 && h0 == last_state) return set_error(SELSCAN_ERR_INVALID_ARG, "h0 and last_state must not alias");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        selscan::DeltaArgs a{};
        a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.lengths = lengths; a.h0 = h0; a.y = y; a.last = last_state;
        a.batch = s->batch; a.L = s->seqlen; a.H = s->nheads; a.P = s->headdim; a.G = s->ngroups;
        a.N = (int)s->dstate; a.scale = scale;
        const int in_bf16 = s->in_dtype == SELSCAN_BF16, out_bf16 = s->out_dtype == SELSCAN_BF16;
        hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
        if (s->seqlen <= kRecTokens) {
            a.vec = vec4(s, q, k) && aligned16(h0) && aligned16(last_state);
            return launched(selscan::launch_delta_rec(a, in_bf16, out_bf16, hs));
        }
        Scratch ws;
        st = ws.get(s->workspace, s->workspace_bytes, fwd_bytes(s), hs);
        if (st != SELSCAN_OK) return st;
        Scratch pad;
        char* recs = static_cast<char*>(ws.ptr);
        st = pad_rows(a, s, recs + record_bytes(s), pad, hs);
        hipError_t e = hipSuccess;
        if (st == SELSCAN_OK) e = selscan::launch_delta_prep(a, in_bf16, false, recs, hs);
        if (st == SELSCAN_OK && e == hipSuccess) e = selscan::launch_delta_scan(a, in_bf16, out_bf16, recs, hs);
        pad.release();
        ws.release();
        return st != SELSCAN_OK ? st : launched(e);
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

size_t selscan_delta_bwd_workspace_bytes(const selscan_m2_shape_t* s) {
    if (check_bwd_shape(s) != SELSCAN_OK) return 0;
    return bwd_bytes(s);
}

selscan_status_t selscan_delta_bwd(const selscan_m2_shape_t* s, const void* q, const void* k, const void* v,
                                   const float* g, const float* beta, float scale, const int32_t* lengths,
                                   const float* h0, const void* dout, const float* dlast_state, void* dq, void* dk,
                                   void* dv, float* dg, float* dbeta, float* dh0, void* stream) {
    try {
        selscan_status_t st = check_bwd_shape(s);
        if (st != SELSCAN_OK) return st;
        if (!q || !k || !v || !g || !beta || !dout)
            return set_error(SELSCAN_ERR_INVALID_ARG, "q, k, v, g, beta and dout must be non-NULL");
        if (!dq || !dk || !dv || !dg || !dbeta)
            return set_error(SELSCAN_ERR_INVALID_ARG, "dq, dk, dv, dg and dbeta must be non-NULL");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
        Scratch ws;
        st = ws.get(s->workspace, s->workspace_bytes, bwd_bytes(s), hs);
        if (st != SELSCAN_OK) return st;
        selscan::DeltaBwdArgs a{};
        a.f.q = q; a.f.k = k; a.f.v = v; a.f.g = g; a.f.beta = beta; a.f.lengths = lengths; a.f.h0 = h0;
        a.f.batch = s->batch; a.f.L = s->seqlen; a.f.H = s->nheads; a.f.P = s->headdim; a.f.G = s->ngroups;
        a.f.N = (int)s->dstate; a.f.scale = scale;
        a.vec_g = s->dstate % 8 == 0 && aligned16(dq) && aligned16(dk);
        a.vec_p = s->headdim % 8 == 0 && aligned16(dout) && aligned16(v);
        a.dout = dout; a.dlast = dlast_state; a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
        selscan::delta_bwd_carve(a, ws.ptr);
        Scratch pad;
        st = pad_rows(a.f, s, static_cast<char*>(ws.ptr) + bwd_main_bytes(s), pad, hs);
        hipError_t e = hipSuccess;
        if (st == SELSCAN_OK)
            e = selscan::launch_delta_bwd(a, s->in_dtype == SELSCAN_BF16, s->out_dtype == SELSCAN_BF16, hs);
        pad.release();
        ws.release();
        return st != SELSCAN_OK ? st : launched(e);
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

selscan_status_t selscan_delta_step(const selscan_m2_shape_t* s, float* state, const void* q, const void* k,
                                    const void* v, const float* g, const float* beta, float scale, void* y,
                                    void* stream) {
    try {
        if (!s) return set_error(SELSCAN_ERR_INVALID_ARG, "shape is NULL");
        selscan_m2_shape_t one = *s;
        one.seqlen = 1;
        selscan_status_t st = check_shape(&one);
        if (st != SELSCAN_OK) return st;
        if (!state || !q || !k || !v || !g || !beta || !y)
            return set_error(SELSCAN_ERR_INVALID_ARG, "state, q, k, v, g, beta and y must be non-NULL");
        if (s->dstate % 4 == 0 && !aligned16(state))
            return set_error(SELSCAN_ERR_INVALID_ARG, "state must be 16-byte aligned");
        st = device_check();
        if (st != SELSCAN_OK) return st;
        selscan::DeltaArgs a{};
        a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.h0 = state; a.y = y; a.last = state;
        a.batch = s->batch; a.L = 1; a.H = s->nheads; a.P = s->headdim; a.G = s->ngroups;
        a.N = (int)s->dstate; a.scale = scale;
        a.vec = vec4(s, q, k);
        return launched(selscan::launch_delta_rec(a, s->in_dtype == SELSCAN_BF16, s->out_dtype == SELSCAN_BF16,
                                                  reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return set_error(SELSCAN_ERR_LAUNCH, "unexpected host exception");
    }
}

}  // extern "C"
