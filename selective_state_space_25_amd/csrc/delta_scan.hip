// delta_scan.hip -- the gated delta rule over 64-token chunks.
//
// With S [N, P] the state entering a chunk, cum the running sum of g inside
// it, and T, A from delta_prep.hip, the chunk's errors, outputs and next
// state are
//
//   R = beta (V - e^cum (K S));   U = T R
//   Y = scale (e^cum (Q S) + A U)
//   S' = e^last S + K^T (e^(last - cum) U)
//
// which is the token recurrence regrouped: U's rows are the u_t of
// S_t = e^g_t S_{t-1} + k_t u_t^T.  Value columns are independent, so a wave
// owns 16 columns of one head and walks its chunks in order with nothing to
// exchange: S, R and U stay in its registers as C tiles, and a C tile pair is
// the B operand of the next product (split_tiles).  A workgroup's waves share
// the chunk's K, Q, T and A in LDS, fetched a chunk ahead.
//
// Products are fp32-grade (split_mfma.hpp) where they reach the state.  What
// goes into a bf16 y alone (Q S, A U) keeps plane pairs a + b < 2, an error
// near 2^-16 under the 2^-9 of y's own rounding.
#include "delta_chunk.hpp"

namespace selscan {

namespace {

using namespace dchunk;

// OL: plane pairs a + b < OL in the products of y; without y (OL = 0) Q and
// A stay out.
template <typename Tin, int NP, int OL>
struct ScanSmem {
    static constexpr int kRow = NP + 8;
    float gam[kC], tail[kC], beta[kC];
    uint16_t K[kPlanes<Tin>][kC][kRow];   // columns through kperm
    Frags<3> T;
    uint16_t Q[OL ? kPlanes<Tin> : 1][OL ? kC : 1][kRow];
    Frags<OL ? OL : 1> A;
};

// KEEP: instead of y, the state entering each chunk [chunk, pad, NP] and U
// [chunk, 64, pad], which the gradients read (pad: P rounded up to 32, the
// columns past P zero).
template <typename Tin, typename Tout, int NP, int W, bool KEEP>
__global__ __launch_bounds__(64 * W) void delta_scan_kernel(DeltaArgs a, const float* recs, int64_t nch, int npb,
                                                            float* keep_s, float* keep_u, int pad) {
    constexpr int OL = KEEP ? 0 : sizeof(Tout) == 2 ? 2 : 3;
    constexpr int NK = kPlanes<Tin>;
    constexpr int kRow = ScanSmem<Tin, NP, OL>::kRow;
    constexpr int NB = NP / 16;              // state tiles
    constexpr int KS = NP / 32;              // k-steps over the key dimension
    constexpr int kT = 64 * W;
    constexpr int NPC = kC * (NP / 8) / kT;  // 8-element pieces of K (or Q) per thread
    constexpr int NTR = (kBlocks * 64 + kT - 1) / kT;   // float4 pieces of T (or A) per thread
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<ScanSmem<Tin, NP, OL>*>(smem_raw);
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    // the column blocks of a head on one XCD (workgroups go round the eight),
    // whose L2 then serves its K, Q and records once from memory
    const int64_t j = blockIdx.x / 8;
    const int64_t bh = (j / npb) * 8 + blockIdx.x % 8;
    if (bh >= a.batch * a.H) return;
    const int64_t b = bh / a.H, h = bh - b * a.H, grp = h / (a.H / a.G);
    const int64_t len = seq_len(a, b);
    const int64_t mine = (len + kC - 1) / kC;
    const int64_t p0 = (int64_t)(j % npb) * 16 * W + 16 * wave;
    const int64_t p = p0 + li;
    const bool active = p0 < (KEEP ? (int64_t)pad : a.P), pok = p < a.P;
    const int N = a.N;
    const Tin* Kg = reinterpret_cast<const Tin*>(a.k);
    const Tin* Qg = reinterpret_cast<const Tin*>(a.q);
    const Tin* Vg = reinterpret_cast<const Tin*>(a.v);
    Tout* Yg = reinterpret_cast<Tout*>(a.y);

    f32x4 S[NB];   // tile i: rows n = 16 i + 4 lg + q, column p
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = 16 * i + 4 * lg + q;
            S[i][q] = a.h0 && pok && n < N ? a.h0[(bh * a.P + p) * N + n] : 0.0f;
        }

    Raw8<Tin> sk[NPC], sq[NPC];   // the next chunk's pieces, on their way to LDS
    float4 stt[NTR], sa[NTR], sgate;
    Tin sv[16];
    auto fetch = [&](int64_t c) {
        const int64_t t0 = c * kC;
        const int live = (int)min((int64_t)kC, len - t0);
        const float* rec = recs + (bh * nch + c) * kRec;
#pragma unroll
        for (int i = 0; i < NPC; ++i) {
            const int id = tid + i * kT, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            if (r < live) {
                const int64_t row = ((b * a.L + t0 + r) * a.G + grp) * N;
                fetch8(Kg + row, n0, N, a.vec, sk[i]);
                if constexpr (!KEEP) fetch8(Qg + row, n0, N, a.vec, sq[i]);
            } else {
                zero(sk[i]);
                if constexpr (!KEEP) zero(sq[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NTR; ++i) {
            const int id = tid + i * kT;
            if (id < kBlocks * 64) {
                const int o = (id >> 6) * 256 + (id & 15) * 16 + ((id >> 4) & 3) * 4;
                stt[i] = *reinterpret_cast<const float4*>(rec + kRecT + o);
                if constexpr (!KEEP) sa[i] = *reinterpret_cast<const float4*>(rec + kRecA + o);
            }
        }
        if (tid < 48) sgate = *reinterpret_cast<const float4*>(rec + kRecGam + 4 * tid);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = 16 * (i >> 2) + 4 * lg + (i & 3);
            sv[i] = pok && r < live ? Vg[((b * a.L + t0 + r) * a.H + h) * a.P + p] : Tin(0);
        }
    };
    auto stage = [&]() {
#pragma unroll
        for (int i = 0; i < NPC; ++i) {
            const int id = tid + i * kT, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            stage8<true>(sm.K[0][r], kC * kRow, n0, sk[i]);
            if constexpr (!KEEP) stage8<true>(sm.Q[0][r], kC * kRow, n0, sq[i]);
        }
#pragma unroll
        for (int i = 0; i < NTR; ++i) {
            const int id = tid + i * kT;
            if (id < kBlocks * 64) {
                int tb, sb;
                lower_tile(id >> 6, tb, sb);
                const int f = frag(tb, sb >> 1), e = 4 * (sb & 1);
                const float tv[4] = {stt[i].x, stt[i].y, stt[i].z, stt[i].w};
                uint2 tp[3];
                split4<3>(tv, tp);
#pragma unroll
                for (int x = 0; x < 3; ++x) *reinterpret_cast<uint2*>(&sm.T.p[x][f][id & 63][e]) = tp[x];
                if constexpr (!KEEP) {
                    const float av[4] = {sa[i].x, sa[i].y, sa[i].z, sa[i].w};
                    uint2 ap[OL];
                    split4<OL>(av, ap);
#pragma unroll
                    for (int x = 0; x < OL; ++x) *reinterpret_cast<uint2*>(&sm.A.p[x][f][id & 63][e]) = ap[x];
                }
            }
        }
        if (tid < 48) *reinterpret_cast<float4*>(&sm.gam[4 * tid]) = sgate;   // gam, tail, beta in a row
    };
    // the zero blocks above the diagonal inside fragments 0 and 3, written once
    for (int i = tid; i < 128; i += kT) {
        const int f = i < 64 ? 0 : 3;
        const uint2 z = make_uint2(0, 0);
#pragma unroll
        for (int x = 0; x < 3; ++x) *reinterpret_cast<uint2*>(&sm.T.p[x][f][i & 63][4]) = z;
        if constexpr (!KEEP) {
#pragma unroll
            for (int x = 0; x < OL; ++x) *reinterpret_cast<uint2*>(&sm.A.p[x][f][i & 63][4]) = z;
        }
    }
    if (mine > 0) {
        fetch(0);
        stage();
    }
    __syncthreads();
    for (int64_t c = 0; c < mine; ++c) {
        const int64_t t0 = c * kC;
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = io::ld(&sv[i]);
        if (c + 1 < mine) fetch(c + 1);
        if (active) {
            bf16x8 Sp[KS][3];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) split_tiles<3>(S[2 * ks], S[2 * ks + 1], Sp[ks]);
            f32x4 R[4], U[4];
            bf16x8 Bp[2][3];
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    bf16x8 k[NK];
#pragma unroll
                    for (int x = 0; x < NK; ++x) k[x] = ld8(&sm.K[x][16 * tb + li][32 * ks + 8 * lg]);
                    acc = mm<3>(k, Sp[ks], acc);
                }
                const f32x4 gam = *reinterpret_cast<const f32x4*>(&sm.gam[16 * tb + 4 * lg]);
                const f32x4 beta = *reinterpret_cast<const f32x4*>(&sm.beta[16 * tb + 4 * lg]);
#pragma unroll
                for (int q = 0; q < 4; ++q) R[tb][q] = beta[q] * __builtin_fmaf(-gam[q], acc[q], v[4 * tb + q]);
            }
            split_tiles<3>(R[0], R[1], Bp[0]);
            split_tiles<3>(R[2], R[3], Bp[1]);
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                U[tb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int ks = 0; ks <= tb / 2; ++ks) {
                    bf16x8 t[3];
                    ld_frag(sm.T, frag(tb, ks), lane, t);
                    U[tb] = mm<3>(t, Bp[ks], U[tb]);
                }
            }
            if constexpr (KEEP) {
                float* ku = keep_u + (bh * nch + c) * kC * pad + p;
#pragma unroll
                for (int i = 0; i < 16; ++i) ku[(16 * (i >> 2) + 4 * lg + (i & 3)) * pad] = U[i >> 2][i & 3];
                float* ks = keep_s + ((bh * nch + c) * pad + p) * NP + 4 * lg;
#pragma unroll
                for (int i = 0; i < NB; ++i) *reinterpret_cast<f32x4*>(ks + 16 * i) = S[i];
            } else {
                // y
                split_tiles<3>(U[0], U[1], Bp[0]);
                split_tiles<3>(U[2], U[3], Bp[1]);
#pragma unroll
                for (int tb = 0; tb < 4; ++tb) {
                    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        bf16x8 x[NK];
#pragma unroll
                        for (int i = 0; i < NK; ++i) x[i] = ld8(&sm.Q[i][16 * tb + li][32 * ks + 8 * lg]);
                        acc = mm<OL>(x, Sp[ks], acc);
                    }
                    acc *= *reinterpret_cast<const f32x4*>(&sm.gam[16 * tb + 4 * lg]);
#pragma unroll
                    for (int ks = 0; ks <= tb / 2; ++ks) {
                        bf16x8 x[OL];
                        ld_frag(sm.A, frag(tb, ks), lane, x);
                        acc = mm<OL>(x, Bp[ks], acc);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int64_t t = t0 + 16 * tb + 4 * lg + q;
                        if (pok && t < a.L) io::st(Yg + ((b * a.L + t) * a.H + h) * a.P + p, a.scale * acc[q]);
                    }
                }
            }
            // the next state
            const float gl = sm.gam[kC - 1];
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) U[tb] *= *reinterpret_cast<const f32x4*>(&sm.tail[16 * tb + 4 * lg]);
            split_tiles<3>(U[0], U[1], Bp[0]);
            split_tiles<3>(U[2], U[3], Bp[1]);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                S[i] *= gl;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    bf16x8 k[NK];
#pragma unroll
                    for (int x = 0; x < NK; ++x) k[x] = ld_down<true>(&sm.K[x][0][0], kRow, 32 * ks, 16 * i, lane);
                    S[i] = mm<3>(k, Bp[ks], S[i]);
                }
            }
        }
        __syncthreads();
        if (c + 1 < mine) stage();
        __syncthreads();
    }
    if (!KEEP && pok) {
        for (int64_t t = mine * kC + lg; t < a.L; t += 4) io::st(Yg + ((b * a.L + t) * a.H + h) * a.P + p, 0.0f);
        if (a.last) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = 16 * i + 4 * lg + q;
                    if (n < N) a.last[(bh * a.P + p) * N + n] = S[i][q];
                }
        }
    }
}

template <typename Tin, typename Tout, int NP, bool KEEP>
hipError_t launch(const DeltaArgs& a, const float* recs, float* keep_s, float* keep_u, int pad, hipStream_t stream) {
    constexpr int W = 4;
    constexpr int bytes = (int)sizeof(ScanSmem<Tin, NP, KEEP ? 0 : sizeof(Tout) == 2 ? 2 : 3>);
    const auto kern = &delta_scan_kernel<Tin, Tout, NP, W, KEEP>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const int npb = (int)((a.P + 16 * W - 1) / (16 * W));
    const int64_t units = (a.batch * a.H + 7) / 8 * 8;
    KTime kt(KEEP ? "delta_keep" : "delta_scan", stream);
    hipLaunchKernelGGL(kern, dim3((unsigned)(units * npb)), dim3(64 * W), bytes, stream, a, recs, delta_chunks(a.L), npb,
                       keep_s, keep_u, pad);
    return hipGetLastError();
}

template <typename Tin, typename Tout>
hipError_t by_n(const DeltaArgs& a, const float* recs, hipStream_t stream) {
    return a.N <= 64 ? launch<Tin, Tout, 64, false>(a, recs, nullptr, nullptr, 0, stream)
                     : launch<Tin, Tout, 128, false>(a, recs, nullptr, nullptr, 0, stream);
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs& a, int in_bf16, int out_bf16, const float* recs, hipStream_t stream) {
    if (in_bf16) return out_bf16 ? by_n<uint16_t, uint16_t>(a, recs, stream) : by_n<uint16_t, float>(a, recs, stream);
    return out_bf16 ? by_n<float, uint16_t>(a, recs, stream) : by_n<float, float>(a, recs, stream);
}

hipError_t launch_delta_keep(const DeltaArgs& a, int in_bf16, const float* recs, float* keep_s, float* keep_u, int pad,
                             hipStream_t stream) {
    if (in_bf16) return a.N <= 64 ? launch<uint16_t, float, 64, true>(a, recs, keep_s, keep_u, pad, stream)
                                  : launch<uint16_t, float, 128, true>(a, recs, keep_s, keep_u, pad, stream);
    return a.N <= 64 ? launch<float, float, 64, true>(a, recs, keep_s, keep_u, pad, stream)
                     : launch<float, float, 128, true>(a, recs, keep_s, keep_u, pad, stream);
}

}  // namespace selscan
