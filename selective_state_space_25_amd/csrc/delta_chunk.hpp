// delta_chunk.hpp -- what the chunked gated delta rule's kernels share: the
// per-chunk record, 64-token staging, and the fragments of triangular
// matrices in LDS.
#pragma once

#include "io.hpp"
#include "kernels.hpp"
#include "split_mfma.hpp"

namespace selscan {
namespace dchunk {

using namespace smm;

constexpr int kC = 64;             // tokens per chunk
constexpr int kBlocks = 10;        // 16 x 16 blocks on and below a chunk matrix's diagonal

// Record of one (batch, head, chunk), in floats: T and A as 10 row-major
// 16 x 16 blocks (block (t, s) at t (t + 1) / 2 + s), then per token
// e^cum, e^(last - cum), beta (zero past the sequence's end), and cum itself
// as doubles.
constexpr int kRecT = 0;
constexpr int kRecA = kBlocks * 256;
constexpr int kRecGam = 2 * kBlocks * 256;
constexpr int kRecTail = kRecGam + kC;
constexpr int kRecBeta = kRecTail + kC;
constexpr int kRecCum = kRecBeta + kC;
constexpr int kRec = kRecCum + 2 * kC;

__device__ __forceinline__ int64_t seq_len(const DeltaArgs& a, int64_t b) {
    return a.lengths ? min((int64_t)max(a.lengths[b], 0), a.L) : a.L;
}

__device__ __forceinline__ float exp_f32(float x) { return fast_exp2(x * kLog2e); }

// Planes that an input of type T takes.
template <typename T> constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;

// Eight elements of a row as loaded.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { uint4 w; };
template <> struct Raw8<float> { float4 lo, hi; };

__device__ __forceinline__ void zero(Raw8<uint16_t>& r) { r.w = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero(Raw8<float>& r) { r.lo = r.hi = make_float4(0, 0, 0, 0); }

// Elements n0 .. n0 + 7 of a row of N (zeros past it); vec: 16-byte loads
// are aligned and N % 8 == 0.
__device__ __forceinline__ void fetch8(const uint16_t* row, int n0, int N, int vec, Raw8<uint16_t>& r) {
    if (vec) {
        if (n0 < N) r.w = *reinterpret_cast<const uint4*>(row + n0);
        else zero(r);
    } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = n0 + i < N ? row[n0 + i] : 0u;
        r.w = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    }
}
__device__ __forceinline__ void fetch8(const float* row, int n0, int N, int vec, Raw8<float>& r) {
    if (vec) {
        if (n0 < N) {
            r.lo = *reinterpret_cast<const float4*>(row + n0);
            r.hi = *reinterpret_cast<const float4*>(row + n0 + 4);
        } else {
            zero(r);
        }
    } else {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = n0 + i < N ? row[n0 + i] : 0.0f;
        r.lo = make_float4(e[0], e[1], e[2], e[3]);
        r.hi = make_float4(e[4], e[5], e[6], e[7]);
    }
}

// Eight elements into the planes of a staged row (plane stride ps elements),
// columns n0 .. n0 + 7, through kperm when PERM.
template <bool PERM>
__device__ __forceinline__ void stage8(uint16_t* row, int ps, int n0, const Raw8<uint16_t>& r) {
    if constexpr (PERM) {
        *reinterpret_cast<uint2*>(row + kperm(n0)) = make_uint2(r.w.x, r.w.y);
        *reinterpret_cast<uint2*>(row + kperm(n0 + 4)) = make_uint2(r.w.z, r.w.w);
    } else {
        *reinterpret_cast<uint4*>(row + n0) = r.w;
    }
}
template <bool PERM>
__device__ __forceinline__ void stage8(uint16_t* row, int ps, int n0, const Raw8<float>& r) {
    const float a[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w}, b[4] = {r.hi.x, r.hi.y, r.hi.z, r.hi.w};
    uint2 pa[3], pb[3];
    split4<3>(a, pa);
    split4<3>(b, pb);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        *reinterpret_cast<uint2*>(row + p * ps + (PERM ? kperm(n0) : n0)) = pa[p];
        *reinterpret_cast<uint2*>(row + p * ps + (PERM ? kperm(n0 + 4) : n0 + 4)) = pb[p];
    }
}

// Tile k of the 10 lower tiles: row block tb, column block sb.
__device__ __forceinline__ void lower_tile(int k, int& tb, int& sb) {
    tb = k >= 6 ? 3 : k >= 3 ? 2 : k >= 1 ? 1 : 0;
    sb = k - tb * (tb + 1) / 2;
}

// A lower triangular chunk matrix as MFMA operands: fragment (row block tb,
// k-step ks <= tb / 2) holds column blocks 2 ks and 2 ks + 1 in
// split_tiles' k order.
__device__ __forceinline__ int frag(int tb, int ks) { return tb < 2 ? tb : 2 * tb - 2 + ks; }

// Its transpose: fragment (row block jb, k-step ks >= jb / 2).
__device__ __forceinline__ int frag_t(int jb, int ks) { return jb < 2 ? 2 * jb + ks : jb + 2; }

// NPL planes of a chunk matrix's six fragments.
template <int NPL>
struct Frags {
    uint16_t p[NPL][6][64][8];
};

template <int NPL>
__device__ __forceinline__ void ld_frag(const Frags<NPL>& f, int i, int lane, bf16x8 (&a)[NPL]) {
#pragma unroll
    for (int p = 0; p < NPL; ++p) a[p] = ld8(f.p[p][i][lane]);
}

}  // namespace dchunk
}  // namespace selscan
