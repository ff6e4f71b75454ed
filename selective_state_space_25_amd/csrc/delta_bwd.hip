// delta_bwd.hip -- gradients of the gated delta rule over 64-token chunks.
//
// With the names of delta_scan.hip, dO = scale dout, D the adjoint of the
// state S' that leaves a chunk, G[t, s] = e^(cum_t - cum_s):
//
//   dU = A^T dO + e^(last - cum) (K D);   dR = T^T dU;   dV = beta dR
//   D_in = e^last D + Q^T (e^cum dO) - K^T (beta e^cum dR)
//
//   X  = (dO U^T) G on and below the diagonal;  E = -beta (dR U^T) G below it
//   dQ = e^cum dO S^T + X K
//   dK = e^(last - cum) U D^T - beta e^cum dR S^T + X^T Q + E K + E^T K
//   beta dbeta = beta (dR.V - e^cum k.(S dR)) + rowsum(E KK^T)
//
// and for the decays, where Z = X QK^T + E KK^T (pairs of different tokens),
// a_t = e^cum (q.(S dO) - beta k.(S dR)), b_t = e^(last - cum) k.(D U):
//
//   dg_t = sum_{i >= t} (rowsum Z - colsum Z + a)_i + sum_{i < t} b_i + e^last <S, D>
//
// Row and column sums are taken of the same Z and, like the dots, in fp64:
// where a key is written over, dg is a small difference of these sums.
//
// Five kernels: the records (delta_prep.hip), the scan that keeps every S
// and U (delta_scan.hip), the scan back over the chunks that makes D, dR and
// dV (16 or 32 value columns a workgroup), the gradients that are local to a
// chunk (all chunks at once), and, where heads share q and k, their sum over
// the heads in a fixed order.  All products are fp32-grade, whatever the
// inputs' type: bf16 gradients are the fp32 ones rounded.
//
// Measured at batch 4, 16 heads of 128 x 128, L 2048, bf16: records 38 us,
// kept scan 87, scan back 143 (0.39 GB, 2.7 TB/s: a chain of three products
// a chunk, 4.5 us), gradients 201 (0.5 GB, 2.5 TB/s), 470 in all; fp32: 50,
// 161, 252 and 248.  Of a workgroup's time in the last, 60 % are the steps over
// the value columns, at the rate of their loads, 20 % the pairs and fp64 dots,
// 10 % the products with X and E; a CU holds one such workgroup, whose LDS (93
// KB) leaves no room for another to load meanwhile.
#include "delta_chunk.hpp"
#include "host.hpp"

namespace selscan {

namespace {

using namespace dchunk;

// ------------------------------------------------------------ the scan back
// Waves share the work as in delta_scan.hip: of the state waves, wave w has
// dU, dR and dV of the tokens 16 w .. 16 w + 15 and a quarter of D's rows; the
// helper wave beside it makes what does not wait for D, A^T dO of the next
// chunk and Q^T (e^cum dO), which it hands over as C tiles, and stages K, Q,
// the gates and dO, a chunk ahead.
constexpr int kBackThreads = 512;

template <typename Tin, typename Tdo, int NP, int CT>
struct BackSmem {
    static constexpr int kRow = NP + 8;
    static constexpr int kBufs = kPlanes<Tin> == 1 ? 2 : 1;   // K by chunk parity, where there is room
    float gate[3][kC];                       // e^cum, e^(last - cum), beta
    uint16_t K[kBufs][kPlanes<Tin>][kC][kRow];
    uint16_t Q[kPlanes<Tin>][kC][kRow];
    Operands<NP / 32, 3> D[CT];
    Operands<2, kPlanes<Tdo>> O[CT];         // dout
    Operands<2, 3> U[CT], R[CT], G[CT];      // dU; -beta e^cum dR; e^cum dO
    Tiles X[CT];                             // A^T dO
    Tiles H[CT][NP / 64];                    // Q^T (e^cum dO): tile i of wave w at [i][w]
};

template <typename Tin, typename Tdo, int NP, int CT>
__global__ __launch_bounds__(kBackThreads, 2) void delta_back_kernel(DeltaBwdArgs ba, int64_t nch, int npb) {
    constexpr int NK = kPlanes<Tin>, NO = kPlanes<Tdo>;
    constexpr int ES = (int)sizeof(Tin), EO = (int)sizeof(Tdo);
    using Smem = BackSmem<Tin, Tdo, NP, CT>;
    constexpr int kRow = Smem::kRow;
    constexpr bool one = Smem::kBufs == 1;
    constexpr int KS = NP / 32, NT = NP / 64, NPC = NP / 32;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<Smem*>(smem_raw);
    const DeltaArgs& a = ba.f;
    const int tid = threadIdx.x & 255, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool helper = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0;
    const int jx = blockIdx.x / 8;
    const int64_t bh = (int64_t)(jx / npb) * 8 + blockIdx.x % 8;
    if (bh >= a.batch * a.H) return;
    const int64_t b = bh / a.H, h = bh - b * a.H, grp = h / (a.H / a.G);
    const int64_t len = seq_len(a, b);
    const Chunks seq(len), all(a.L);
    const int mine = seq.n;
    const int N = a.N, P = (int)a.P, pad = ba.pad;
    const int p0 = (jx % npb) * 16 * CT + li;
    const int sv = scalar((int)(a.H * P * ES));
    char* dVg = scalar(static_cast<char*>(ba.dv) + b * a.L * sv + h * P * ES);
    const char* Rg = scalar(ba.recs + bh * nch * GradRec::bytes);
    const f32x4 z4 = {0.0f, 0.0f, 0.0f, 0.0f};
    auto record = [&](int c) { return rows_buf(Rg + (int64_t)c * GradRec::bytes, c < 0 ? 0 : 1, 0, GradRec::bytes); };
    int toff[2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) toff[ks] = row_of_t(w, ks, lane);
    // Inputs are asked for as soon as the chunk before has used their
    // registers, a chunk's work ahead (before the first chunk: buffers of no
    // rows)
    bf16x8 fm[2][3];   // T^T for a state wave, A^T for a helper
    auto fetch_m = [&](int c, int at) {
        const auto rb = record(c);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int x = 0; x < 3; ++x) fm[ks][x] = buf_op(rb, toff[ks] + at + x * kPlane);
    };

    if (!helper) {
        f32x4 D[NT][CT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = 16 * (NT * w + i) + 4 * lg + q, p = p0 + 16 * ct;
                    D[i][ct][q] = ba.dlast && p < P && n < N ? ba.dlast[(bh * P + p) * N + n] : 0.0f;
                }
        auto put_state = [&]() {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < NT; ++i) sm.D[ct].put_tile(NT * w + i, D[i][ct], lane);
        };
        int voff[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const int p = p0 + 16 * ct;
            voff[ct] = p < P ? (16 * w + 4 * lg) * sv + p * ES : kOut;
        }
        fetch_m(mine - 1, GradRec::Tt);
        put_state();
        lds_barrier();
        lds_barrier();
        for (int c = mine - 1; c >= 0; --c) {
            const uint16_t* K = &sm.K[one ? 0 : c & 1][0][0][0];
            // dU for the wave's tokens
            auto gate = [&](int i) { return *reinterpret_cast<const f32x4*>(sm.gate[i] + 16 * w + 4 * lg); };
            const f32x4 gam = gate(0), tail = gate(1), beta = gate(2);
            const float gl = sm.gate[0][kC - 1];
            {
                bf16x8 k[KS][NK];
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int x = 0; x < NK; ++x) k[ks][x] = ld8(K + (x * kC + 16 * w + li) * kRow + 32 * ks + 8 * lg);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    bf16x8 d[KS][3];
                    f32x4 acc[KS];
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        sm.D[ct].get(ks, lane, d[ks]);
                        acc[ks] = z4;
                    }
                    mm_turns<3, NK, 3>([&](int m) { return k[m]; }, [&](int m) { return d[m]; }, acc);
                    sm.U[ct].put_tile(w, sum_of(acc) * tail + sm.X[ct].get(w, lane), lane);
                    float* kd = ba.D + (bh * nch + c) * pad * NP + kept_tile<NP>(p0 - li + 16 * ct, NT * w, lane);
#pragma unroll
                    for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4*>(kd + 256 * i) = D[i][ct];
                }
            }
            lds_barrier();
            // dR and dV for the wave's tokens (the last two waves' rows of
            // T^T begin in the second k-step)
            f32x4 r[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bf16x8 y[2][3];
                sm.U[ct].get(1, lane, y[1]);
                if (w >= 2) {
                    r[ct] = mm<3>(fm[1], y[1], z4);
                } else {
                    sm.U[ct].get(0, lane, y[0]);
                    r[ct] = mm_pair(fm, y);
                }
                sm.R[ct].put_tile(w, -(r[ct] * beta * gam), lane);
            }
            fetch_m(c - 1, GradRec::Tt);
            bf16x8 k[NT * 2][NK];
#pragma unroll
            for (int i = 0; i < NT * 2; ++i)
#pragma unroll
                for (int l = 0; l < NK; ++l)
                    k[i][l] = ld_down(K + l * kC * kRow, kRow, 32 * (i & 1), 16 * (NT * w + i / 2), lane);
            const auto vb = rows_buf(scalar(dVg + (int64_t)c * kC * sv), scalar(all.rows(c)), sv, P * ES);
            const int live = seq.rows(c) - (16 * w + 4 * lg);   // (past the end zero whatever the states hold)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float* kr = ba.dR + (bh * nch + c) * kC * pad + p0 + 16 * ct;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    kr[(16 * w + 4 * lg + q) * pad] = r[ct][q];
                    buf_st(vb, voff[ct] + q * sv, q < live ? beta[q] * r[ct][q] : 0.0f, Tin(0));
                }
            }
            lds_barrier();
            // the wave's rows of the adjoint before the chunk
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bf16x8 y[2][3];
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) sm.R[ct].get(ks, lane, y[ks]);
                f32x4 acc[NT * 2];
#pragma unroll
                for (int i = 0; i < NT * 2; ++i) acc[i] = i & 1 ? sm.H[ct][i / 2].get(w, lane) : D[i / 2][ct] * gl;
                mm_turns<3, NK, 3>([&](int m) { return k[m]; }, [&](int m) { return y[m & 1]; }, acc);
#pragma unroll
                for (int i = 0; i < NT; ++i) D[i][ct] = acc[2 * i] + acc[2 * i + 1];
            }
            put_state();
            lds_barrier();
        }
        if (ba.dh0) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = 16 * (NT * w + i) + 4 * lg + q, p = p0 + 16 * ct;
                        if (p < P && n < N) ba.dh0[(bh * P + p) * N + n] = D[i][ct][q];
                    }
        }
        return;
    }

    // ---- helper waves
    const int sk = scalar((int)(a.G * a.qk_row * ES)), so = scalar((int)(a.H * P * EO));
    const int64_t krow = b * a.L * sk + grp * a.qk_row * ES;
    const char* Kg = scalar(static_cast<const char*>(a.k) + krow);
    const char* Qg = scalar(static_cast<const char*>(a.q) + krow);
    const char* Og = scalar(static_cast<const char*>(ba.dout) + b * a.L * so + h * P * EO);
    int koff[NPC], ooff[CT];
#pragma unroll
    for (int i = 0; i < NPC; ++i) {
        const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
        koff[i] = n0 < a.NL ? r * sk + n0 * ES : kOut;
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int p = p0 + 16 * ct;
        ooff[ct] = p < P ? (16 * w + 4 * lg) * so + p * EO : kOut;
    }
    Raw8<Tin> fk[NPC], fq[NPC];
    f32x4 fgate[3];
    Tdo fo[CT][4];
    auto rows = [&](const char* base, int stride, int c, int bytes) {
        return rows_buf(base + (int64_t)c * kC * stride, c < 0 ? 0 : seq.rows(c), stride, bytes);
    };
    auto fetch_p = [&](const char* base, int c, Raw8<Tin> (&f)[NPC]) {
        const auto kb = rows(base, sk, c, a.NL * ES);
#pragma unroll
        for (int i = 0; i < NPC; ++i) fetch8(kb, koff[i], f[i]);
    };
    auto fetch_o = [&](int c) {   // and the gates of the wave's tokens
        const auto rb = record(c);
#pragma unroll
        for (int i = 0; i < 3; ++i) fgate[i] = buf_ld4(rb, GradRec::gam + (i * kC + 16 * w + 4 * lg) * 4);
        const auto ob = rows(Og, so, c, P * EO);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int q = 0; q < 4; ++q) fo[ct][q] = buf_raw<Tdo>(ob, ooff[ct] + q * so);
    };
    auto stage_p = [&](uint16_t (*m)[kC][kRow], const Raw8<Tin> (&f)[NPC]) {
#pragma unroll
        for (int i = 0; i < NPC; ++i) {
            const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            stage8(m[0][r], kC * kRow, n0, f[i]);
        }
    };
    auto stage_k = [&](int c) {
        stage_p(sm.K[one ? 0 : c & 1], fk);
        fetch_p(Kg, c - 1, fk);
    };
    // all that a chunk needs in LDS but K; and the next one's on the way
    auto stage = [&](int c) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (li == 0) *reinterpret_cast<f32x4*>(sm.gate[i] + 16 * w + 4 * lg) = fgate[i];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const f32x4 o = widen(fo[ct]);
            sm.O[ct].put_tile(w, o, lane);
            sm.G[ct].put_tile(w, o * fgate[0] * a.scale, lane);
        }
        fetch_o(c - 1);
        stage_p(sm.Q, fq);
        fetch_p(Qg, c - 1, fq);
    };
    // A^T dO for the wave's tokens
    auto put_x = [&](int c) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            bf16x8 d[2][NO];
            f32x4 x;
            sm.O[ct].get(1, lane, d[1]);
            if (w >= 2) {
                x = mm<3>(fm[1], d[1], z4);
            } else {
                sm.O[ct].get(0, lane, d[0]);
                f32x4 acc[2] = {z4, z4};
                mm_turns<3, 3, NO>([&](int m) { return fm[m]; }, [&](int m) { return d[m]; }, acc);
                x = sum_of(acc);
            }
            sm.X[ct].put(w, x * a.scale, lane);
        }
        fetch_m(c - 1, GradRec::At);
    };

    {
        const int c = mine - 1;
        fetch_o(c);
        fetch_p(Qg, c, fq);
        fetch_p(Kg, c, fk);
        fetch_m(c, GradRec::At);
        stage(c);
        stage_k(c);
        lds_barrier();
        put_x(c);
        lds_barrier();
    }
    for (int c = mine - 1; c >= 0; --c) {
        // Q^T (e^cum dO), the wave's rows
        {
            bf16x8 q[NT * 2][NK];
#pragma unroll
            for (int i = 0; i < NT * 2; ++i)
#pragma unroll
                for (int l = 0; l < NK; ++l) q[i][l] = ld_down(&sm.Q[l][0][0], kRow, 32 * (i & 1), 16 * (NT * w + i / 2), lane);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bf16x8 g[2][3];
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) sm.G[ct].get(ks, lane, g[ks]);
                f32x4 acc[NT * 2];
#pragma unroll
                for (int i = 0; i < NT * 2; ++i) acc[i] = z4;
                mm_turns<3, NK, 3>([&](int m) { return q[m]; }, [&](int m) { return g[m & 1]; }, acc);
#pragma unroll
                for (int i = 0; i < NT; ++i) sm.H[ct][i].put(w, acc[2 * i] + acc[2 * i + 1], lane);
            }
        }
        lds_barrier();
        stage(c - 1);
        if constexpr (!one) stage_k(c - 1);
        lds_barrier();
        put_x(c - 1);
        // (the state waves have K in registers since the barrier)
        if constexpr (one) stage_k(c - 1);
        lds_barrier();
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
        if (p0 + 16 * ct < P)
            for (int64_t t = (int64_t)mine * kC + 4 * w + lg; t < a.L; t += 16)
                io::st(reinterpret_cast<Tin*>(dVg + t * sv) + p0 + 16 * ct, 0.0f);
}

// ------------------------------------------------- gradients inside a chunk
// Eight waves: wave w has the 16 tokens of row block w % 4 and half w / 4 of
// the key's columns; of its row block's pairs it has every other block.
constexpr int kGradThreads = 512;
constexpr int kPb = 32;            // value columns per step of the sums over p
constexpr int kRowP = kPb + 8;
constexpr int kRowX = kC + 8;

template <typename Tin, typename Tdo, int NP>
struct GradSmem {
    static constexpr int kRow = NP + 8;
    double cum[kC];
    double col[4][kC];             // per row block: column sums of Z
    double sd[8];
    float rv[kC];
    union {
        struct {                   // a step over 32 value columns
            uint16_t S[3][kPb][kRow], D[3][kPb][kRow];
            uint16_t U[3][kC][kRowP], R[3][kC][kRowP];
            uint16_t O[kPlanes<Tdo>][kC][kRowP];
        } s;
        struct {                   // the chunk's pairs
            uint16_t K[kPlanes<Tin>][kC][kRow], Q[kPlanes<Tin>][kC][kRow];
            uint16_t X[3][kC][kRowX], E[3][kC][kRowX];
        } m;
    };
    // A half's sums for token t, in the padding of its rows of X and E:
    // rowsum Z + a; b; what dbeta gets beside dR.V.
    __device__ __forceinline__ double* up(int t) { return reinterpret_cast<double*>(&m.X[0][t][kC]); }
    __device__ __forceinline__ double* down(int t) { return reinterpret_cast<double*>(&m.X[1][t][kC]); }
    __device__ __forceinline__ double* db(int t) { return reinterpret_cast<double*>(&m.E[0][t][kC]); }
};

// Four elements of a row as loaded, those past n zero (vec: in one piece).
template <typename T> struct Raw4;
template <> struct Raw4<uint16_t> { unsigned w[2]; };
template <> struct Raw4<float> { f32x4 v; };
__device__ __forceinline__ void fetch4(__amdgpu_buffer_rsrc_t b, int off, int n, int vec, Raw4<uint16_t>& r) {
    if (vec) {
        const auto w = __builtin_amdgcn_raw_buffer_load_b64(b, n > 0 ? off : kOut, 0, 0);
        r.w[0] = w[0];
        r.w[1] = w[1];
    } else {
        unsigned e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = __builtin_amdgcn_raw_buffer_load_b16(b, i < n ? off + 2 * i : kOut, 0, 0);
        r.w[0] = e[0] | e[1] << 16;
        r.w[1] = e[2] | e[3] << 16;
    }
}
__device__ __forceinline__ void fetch4(__amdgpu_buffer_rsrc_t b, int off, int n, int vec, Raw4<float>& r) {
    if (vec) {
        r.v = buf_ld4(b, n > 0 ? off : kOut);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[i] = buf_raw<float>(b, i < n ? off + 4 * i : kOut);
    }
}
__device__ __forceinline__ f32x4 widen(const Raw4<uint16_t>& r) {
    return f32x4{bf16lo(r.w[0]), bf16hi(r.w[0]), bf16lo(r.w[1]), bf16hi(r.w[1])};
}
__device__ __forceinline__ f32x4 widen(const Raw4<float>& r) { return r.v; }

// The value of the lane that a data-parallel move names.
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)w, CTRL, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(w >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over 16 lanes, in every one of them: over pairs, pairs of pairs (lanes
// exchanged within four), the halves of eight and of sixteen (mirrored).
__device__ __forceinline__ double sum16(double v) {
    v += moved<0xB1>(v);
    v += moved<0x4E>(v);
    v += moved<0x141>(v);
    v += moved<0x140>(v);
    return v;
}

// Into the planes of a staged row (plane stride ps elements).
__device__ __forceinline__ void stage4(uint16_t* row, int ps, const Raw4<uint16_t>& r) {
    *reinterpret_cast<uint2*>(row) = make_uint2(r.w[0], r.w[1]);
}
__device__ __forceinline__ void stage4(uint16_t* row, int ps, const Raw4<float>& r) {
    uint2 p[3];
    split4<3>(r.v, p);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(row + i * ps) = p[i];
}

template <typename Tin, typename Tdo, int NP>
__global__ __launch_bounds__(kGradThreads) void delta_grad_kernel(DeltaBwdArgs ba, int64_t nch) {
    constexpr int NK = kPlanes<Tin>, NO = kPlanes<Tdo>;
    using Smem = GradSmem<Tin, Tdo, NP>;
    constexpr int kRow = Smem::kRow;
    constexpr int NB = NP / 16, NH = NB / 2;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<Smem*>(smem_raw);
    const DeltaArgs& a = ba.f;
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), tb = wave & 3, half = wave >> 2;
    const int64_t bh = blockIdx.x / nch, c = blockIdx.x - bh * nch;
    const int64_t b = bh / a.H, h = bh - b * a.H, grp = h / (a.H / a.G);
    const int64_t t0 = c * kC;
    const int64_t len = seq_len(a, b);
    const int live = (int)max((int64_t)0, min((int64_t)kC, len - t0));
    const int inside = (int)min((int64_t)kC, a.L - t0);   // tokens of the chunk that exist
    const int N = a.N;
    const int pad = ba.pad;
    // dq and dk: one row per head where they are summed over a group later
    const bool shared_qk = ba.pq != nullptr;
    auto put = [&](void* out, float* part, int r, int n, float v) {
        if (shared_qk) part[((b * a.L + t0 + r) * a.H + h) * N + n] = v;
        else io::st(reinterpret_cast<Tin*>(out) + ((b * a.L + t0 + r) * a.G + grp) * N + n, v);
    };
    if (live == 0) {
        for (int i = tid; i < inside * N; i += kGradThreads) {
            put(ba.dq, ba.pq, i / N, i % N, 0.0f);
            put(ba.dk, ba.pk, i / N, i % N, 0.0f);
        }
        if (tid < inside) {
            ba.dg[(b * a.L + t0 + tid) * a.H + h] = 0.0f;
            ba.dbeta[(b * a.L + t0 + tid) * a.H + h] = 0.0f;
        }
        return;
    }
    const char* rec = ba.recs + (int64_t)blockIdx.x * GradRec::bytes;
    if (tid < kC) sm.cum[tid] = reinterpret_cast<const double*>(rec + GradRec::cum)[tid];

    // ---- sums over the value columns: dO S^T, dR S^T, U D^T for the wave's
    // tokens and columns, dO U^T and dR U^T for its pairs, <S, D>, dR.V
    const f32x4 z4 = {0.0f, 0.0f, 0.0f, 0.0f};
    // (U D^T in two sums: D may be far larger than what of it reaches dg)
    f32x4 q1[NH], k2[NH], k3[NH], k3r[NH], x1[2], x2[2];
#pragma unroll
    for (int i = 0; i < NH; ++i) q1[i] = k2[i] = k3[i] = k3r[i] = z4;
#pragma unroll
    for (int i = 0; i < 2; ++i) x1[i] = x2[i] = z4;
    double sd = 0.0;
    float rv = 0.0f;
    const float* Sg = ba.S + (int64_t)blockIdx.x * pad * NP;
    const float* Dg = ba.D + (int64_t)blockIdx.x * pad * NP;
    const float* Ug = ba.U + (int64_t)blockIdx.x * kC * pad;
    const float* Rg = ba.dR + (int64_t)blockIdx.x * kC * pad;
    constexpr int ES = (int)sizeof(Tin), EO = (int)sizeof(Tdo);
    const int P = (int)a.P;
    const int sk = scalar((int)(a.G * a.qk_row * ES)), sv = scalar((int)(a.H * P * ES)), so = scalar((int)(a.H * P * EO));
    const int64_t row0 = b * a.L + t0;
    const auto ob = rows_buf(scalar(static_cast<const char*>(ba.dout) + row0 * so + h * P * EO), scalar(live), so, P * EO);
    const auto vb = rows_buf(scalar(static_cast<const char*>(a.v) + row0 * sv + h * P * ES), scalar(live), sv, P * ES);
    // A step's inputs are fetched while the step before computes.
    f32x4 fs[NP / 64], fd[NP / 64], fu, fr;
    Raw4<Tin> fv;
    Raw4<Tdo> fo;
    const int pr = tid >> 3, pe = 4 * (tid & 7);   // the thread's row and columns of a step's U, dR, V and dO
    auto fetch = [&](int pb) {
#pragma unroll
        for (int i = 0; i < NP / 64; ++i) {      // S and D: two column blocks' tiles in turn
            const int id = wave + 8 * i;
            fs[i] = *reinterpret_cast<const f32x4*>(Sg + kept_tile<NP>(pb + 16 * (id / NB), id % NB, lane));
            fd[i] = *reinterpret_cast<const f32x4*>(Dg + kept_tile<NP>(pb + 16 * (id / NB), id % NB, lane));
        }
        const int e0 = pb + pe;
        fu = *reinterpret_cast<const f32x4*>(Ug + (int64_t)pr * pad + e0);
        fr = *reinterpret_cast<const f32x4*>(Rg + (int64_t)pr * pad + e0);
        fetch4(vb, pr * sv + e0 * ES, P - e0, ba.vec_p, fv);
        fetch4(ob, pr * so + e0 * EO, P - e0, ba.vec_p, fo);
    };
    // what follows the steps: K, Q, and A's rows of the wave's tokens
    Raw8<Tin> fk[NP / 64], fq[NP / 64];
    float am[2][4];
    auto fetch_kq = [&]() {
        const auto rb = rows_buf(scalar(rec), 1, 0, GradRec::bytes);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int sb = 2 * j + half;
                am[j][q] = buf_raw<float>(rb, sb <= tb ? GradRec::A + (block_at(tb, sb) * 256 + (4 * lg + q) * 16 + li) * 4 : kOut);
            }
        const int64_t at = row0 * sk + grp * a.qk_row * ES;
        const auto kb = rows_buf(scalar(static_cast<const char*>(a.k) + at), scalar(live), sk, a.NL * ES);
        const auto qb = rows_buf(scalar(static_cast<const char*>(a.q) + at), scalar(live), sk, a.NL * ES);
#pragma unroll
        for (int i = 0; i < NP / 64; ++i) {
            const int id = tid + kGradThreads * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            const int off = n0 < a.NL ? r * sk + n0 * ES : kOut;
            fetch8(kb, off, fk[i]);
            fetch8(qb, off, fq[i]);
        }
    };
    fetch(0);
    for (int pb = 0; pb < pad; pb += kPb) {
        lds_barrier();
#pragma unroll
        for (int i = 0; i < NP / 64; ++i) {
            const int id = wave + 8 * i, r = 16 * (id / NB) + li, n = 16 * (id % NB) + 4 * lg;
#pragma unroll
            for (int e = 0; e < 4; ++e) sd = __builtin_fma((double)fs[i][e], (double)fd[i][e], sd);
            uint2 sp[3], dp[3];
            split4<3>(fs[i], sp);
            split4<3>(fd[i], dp);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                *reinterpret_cast<uint2*>(&sm.s.S[x][r][n]) = sp[x];
                *reinterpret_cast<uint2*>(&sm.s.D[x][r][n]) = dp[x];
            }
        }
        const f32x4 v = widen(fv);
#pragma unroll
        for (int e = 0; e < 4; ++e) rv = __builtin_fmaf(fr[e], v[e], rv);
        uint2 up[3], dp[3];
        split4<3>(fu, up);
        split4<3>(fr, dp);
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            *reinterpret_cast<uint2*>(&sm.s.U[x][pr][pe]) = up[x];
            *reinterpret_cast<uint2*>(&sm.s.R[x][pr][pe]) = dp[x];
        }
        stage4(&sm.s.O[0][pr][pe], kC * kRowP, fo);
        lds_barrier();
        if (pb + kPb < pad) fetch(pb + kPb);
        else if (NK == 1) fetch_kq();
        bf16x8 o[NO], r[3], u[3];
#pragma unroll
        for (int x = 0; x < NO; ++x) o[x] = ld8(&sm.s.O[x][16 * tb + li][8 * lg]);
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            r[x] = ld8(&sm.s.R[x][16 * tb + li][8 * lg]);
            u[x] = ld8(&sm.s.U[x][16 * tb + li][8 * lg]);
        }
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            bf16x8 s[3], d[3];
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                s[x] = ld_down(&sm.s.S[x][0][0], kRow, 0, 16 * (half * NH + i), lane);
                d[x] = ld_down(&sm.s.D[x][0][0], kRow, 0, 16 * (half * NH + i), lane);
            }
            // the planes' products in turn over the sums
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
                for (int y = 0; y <= x; ++y) {
                    k2[i] = mfma(r[y], s[x - y], k2[i]);
                    if (x > 0) k3r[i] = mfma(u[y], d[x - y], k3r[i]);
                    else k3[i] = mfma(u[0], d[0], k3[i]);
                    if (y < NO) q1[i] = mfma(o[y], s[x - y], q1[i]);
                }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int sb = 2 * j + half;
            if (sb > tb) continue;
            bf16x8 w[3];
#pragma unroll
            for (int x = 0; x < 3; ++x) w[x] = ld8(&sm.s.U[x][16 * sb + li][8 * lg]);
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
                for (int y = 0; y <= x; ++y) {
                    x2[j] = mfma(r[y], w[x - y], x2[j]);
                    if (y < NO) x1[j] = mfma(o[y], w[x - y], x1[j]);
                }
        }
    }
    if (NK != 1) fetch_kq();   // (fp32: no registers for them before)
    // (asked for here, used after the next barrier)
    const f32x4 gam = *reinterpret_cast<const f32x4*>(rec + GradRec::gam + 4 * (16 * tb + 4 * lg));
    const f32x4 tail = *reinterpret_cast<const f32x4*>(rec + GradRec::tail + 4 * (16 * tb + 4 * lg));
    const f32x4 beta = *reinterpret_cast<const f32x4*>(rec + GradRec::beta + 4 * (16 * tb + 4 * lg));
    const int64_t gi = (b * a.L + t0 + lane) * a.H + h;
    const float gown = wave == 0 && lane < inside ? a.g[gi] : 0.0f;
    const float glast = reinterpret_cast<const float*>(rec + GradRec::gam)[kC - 1];
    lds_barrier();
    sd = sum16(sd);
    sd += __shfl_xor(sd, 16, 64);
    sd += __shfl_xor(sd, 32, 64);
    if (lane == 0) sm.sd[wave] = sd;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) rv += __shfl_xor(rv, o, 64);
    if ((tid & 7) == 0) sm.rv[pr] = rv;
    // K and Q over what the steps used
#pragma unroll
    for (int i = 0; i < NP / 64; ++i) {
        const int id = tid + kGradThreads * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
        stage8(sm.m.K[0][r], kC * kRow, n0, fk[i]);
        stage8(sm.m.Q[0][r], kC * kRow, n0, fq[i]);
    }
    __syncthreads();

    // ---- the dots with q and k; dQ and dK from the states
    double aq[4] = {}, ak[4] = {}, bk[4] = {};
#pragma unroll
    for (int i = 0; i < NH; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 16 * tb + 4 * lg + q, n = 16 * (half * NH + i) + li;
            float kv = 0.0f, qv = 0.0f;
#pragma unroll
            for (int x = NK - 1; x >= 0; --x) {
                kv += bf16_to_f32(sm.m.K[x][r][n]);
                qv += bf16_to_f32(sm.m.Q[x][r][n]);
            }
            aq[q] = __builtin_fma((double)qv, (double)q1[i][q], aq[q]);
            ak[q] = __builtin_fma((double)kv, (double)k2[i][q], ak[q]);
            bk[q] = __builtin_fma((double)kv, (double)k3[i][q] + (double)k3r[i][q], bk[q]);
            k3[i][q] += k3r[i][q];
            q1[i][q] *= a.scale * gam[q];
            k3[i][q] = __builtin_fmaf(tail[q], k3[i][q], -beta[q] * gam[q] * k2[i][q]);
        }
    // ---- pairs: X, E and the sums of Z
    double row[4] = {}, rb[4] = {};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float xv[4] = {}, ev[4] = {};
        const int sb = 2 * j + half, s = 16 * sb + li;
        if (sb <= tb) {
            f32x4 kk = z4;
#pragma unroll
            for (int ks = 0; ks < NP / 32; ++ks) {
                bf16x8 x[NK], y[NK];
#pragma unroll
                for (int p = 0; p < NK; ++p) {
                    x[p] = ld8(&sm.m.K[p][16 * tb + li][32 * ks + 8 * lg]);
                    y[p] = ld8(&sm.m.K[p][s][32 * ks + 8 * lg]);
                }
                kk = mm<3>(x, y, kk);
            }
            const double cs = sm.cum[s];
            double cz = 0.0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int t = 16 * tb + 4 * lg + q;
                const float g = s <= t ? exp_f32((float)(sm.cum[t] - cs)) : 0.0f;
                const float gl = s < t ? g : 0.0f;
                const float e0 = -x2[j][q] * gl;             // E without beta
                xv[q] = a.scale * x1[j][q] * g;
                ev[q] = beta[q] * e0;
                const double ekk = (double)e0 * kk[q];
                const double zv = (s < t ? (double)a.scale * x1[j][q] * am[j][q] : 0.0) + beta[q] * ekk;
                rb[q] += ekk;
                row[q] += zv;
                cz += zv;
            }
            cz += __shfl_xor(cz, 16, 64);
            cz += __shfl_xor(cz, 32, 64);
            if (lg == 0) sm.col[tb][s] = cz;
        }
        // (block tb + 1 of an even row block shares its k-step: zero)
        if (sb <= (tb | 1)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int t = 16 * tb + 4 * lg + q;
                float x = xv[q], e = ev[q];
#pragma unroll
                for (int l = 0; l < 3; ++l) {
                    const uint16_t xh = f32_to_bf16(x), eh = f32_to_bf16(e);
                    sm.m.X[l][t][s] = xh;
                    sm.m.E[l][t][s] = eh;
                    x -= bf16_to_f32(xh);
                    e -= bf16_to_f32(eh);
                }
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int t = 16 * tb + 4 * lg + q;
        aq[q] = sum16(aq[q]);
        ak[q] = sum16(ak[q]);
        bk[q] = sum16(bk[q]);
        row[q] = sum16(row[q]);
        rb[q] = sum16(rb[q]);
        if (li == 0) {
            sm.up(t)[half] = row[q] + gam[q] * (a.scale * aq[q] - beta[q] * ak[q]);
            sm.down(t)[half] = tail[q] * bk[q];
            sm.db(t)[half] = rb[q] - gam[q] * ak[q];
        }
    }
    __syncthreads();
    if (wave == 0) {   // dg and dbeta: lane = token
        double up = sm.up(lane)[0] + sm.up(lane)[1], down = sm.down(lane)[0] + sm.down(lane)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= lane / 16) up -= sm.col[i][lane];
        const double own = down;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double u = __shfl_down(up, o, 64), d = __shfl_up(down, o, 64);
            if (lane + o < 64) up += u;
            if (lane >= o) down += d;
        }
        const double last = glast *
                            (((sm.sd[0] + sm.sd[1]) + (sm.sd[2] + sm.sd[3])) + ((sm.sd[4] + sm.sd[5]) + (sm.sd[6] + sm.sd[7])));
        if (lane < inside) {
            // a decay that is zero has no gradient; the sums would leave their rounding
            ba.dbeta[gi] = lane < live ? (float)(sm.rv[lane] + (sm.db(lane)[0] + sm.db(lane)[1])) : 0.0f;
            ba.dg[gi] = lane < live && exp_f32(gown) != 0.0f ? (float)(up + (down - own) + last) : 0.0f;
        }
    }
    // ---- dQ += X K;  dK += X^T Q + E K + E^T K
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const bool lo = ks <= tb / 2, hi = ks >= tb / 2;   // rows of X and E; their columns
        bf16x8 x[3], e[3], xt[3], et[3];
#pragma unroll
        for (int l = 0; l < 3; ++l) {
            if (lo) {
                x[l] = ld8(&sm.m.X[l][16 * tb + li][32 * ks + 8 * lg]);
                e[l] = ld8(&sm.m.E[l][16 * tb + li][32 * ks + 8 * lg]);
            }
            if (hi) {
                xt[l] = ld_down(&sm.m.X[l][0][0], kRowX, 32 * ks, 16 * tb, lane);
                et[l] = ld_down(&sm.m.E[l][0][0], kRowX, 32 * ks, 16 * tb, lane);
            }
        }
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            const int n0 = 16 * (half * NH + i);
            bf16x8 k[NK], q[NK];
#pragma unroll
            for (int p = 0; p < NK; ++p) k[p] = ld_down(&sm.m.K[p][0][0], kRow, 32 * ks, n0, lane);
            if (lo) {
                q1[i] = mm<3>(x, k, q1[i]);
                k3[i] = mm<3>(e, k, k3[i]);
            }
            if (hi) {
#pragma unroll
                for (int p = 0; p < NK; ++p) q[p] = ld_down(&sm.m.Q[p][0][0], kRow, 32 * ks, n0, lane);
                k3[i] = mm<3>(et, k, k3[i]);
                k3[i] = mm<3>(xt, q, k3[i]);
            }
        }
    }
    // rows through LDS (over K and Q), out 32 bytes or more a lane; past the
    // sequence's end zeros, whatever the states hold
    lds_barrier();
    constexpr int NW = NP / 2, nr = NW + 4;
    float (&out)[16][nr] = *reinterpret_cast<float (*)[16][nr]>(&sm.m.K[0][0][0] + wave * (2 * 16 * nr));
    static_assert(8 * 16 * nr * 4 <= (int)sizeof(sm.m.K) + (int)sizeof(sm.m.Q), "the waves' rows fit over K and Q");
    auto put_rows = [&](const f32x4 (&v)[NH], void* to, float* part) {
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) out[4 * lg + q][16 * i + li] = 16 * tb + 4 * lg + q < live ? v[i][q] : 0.0f;
        wave_sync();
        const int rows = min(16, inside - 16 * tb);
        const bool wide = shared_qk ? N % 8 == 0 : ba.vec_g;
        auto each = [&](auto* first, int64_t stride) {   // row r at first + r stride
            if (wide) {
                for (int id = lane; id < 2 * NW; id += 64) {
                    const int r = id / (NW / 8), m = 8 * (id % (NW / 8)), n = half * NW + m;
                    if (r < rows && n < N) io::st8(first + r * stride + n, &out[r][m]);
                }
            } else {
                for (int id = lane; id < 16 * NW; id += 64) {
                    const int r = id / NW, m = id % NW, n = half * NW + m;
                    if (r < rows && n < N) io::st(first + r * stride + n, out[r][m]);
                }
            }
        };
        const int64_t t = row0 + 16 * tb;
        if (shared_qk) each(part + (t * a.H + h) * N, a.H * N);
        else each(reinterpret_cast<Tin*>(to) + (t * a.G + grp) * N, a.G * N);
        wave_sync();
    };
    put_rows(q1, ba.dq, ba.pq);
    put_rows(k3, ba.dk, ba.pk);
}

// dq and dk of a group: the sum over its heads, in their order.
template <typename Tin>
__global__ __launch_bounds__(256) void delta_group_kernel(DeltaBwdArgs ba) {
    const DeltaArgs& a = ba.f;
    const int64_t i = io::group_id() * 256 + threadIdx.x;   // [batch * L, G, N]
    const int64_t n = i % a.N, tg = i / a.N;
    if (tg >= a.batch * a.L * a.G) return;
    const int64_t r = a.H / a.G;
    float q = 0.0f, k = 0.0f;
    for (int64_t j = 0; j < r; ++j) {   // head g r + j of token t is row t H + g r + j = tg r + j
        q += ba.pq[(tg * r + j) * a.N + n];
        k += ba.pk[(tg * r + j) * a.N + n];
    }
    io::st(reinterpret_cast<Tin*>(ba.dq) + i, q);
    io::st(reinterpret_cast<Tin*>(ba.dk) + i, k);
}

template <typename K>
hipError_t lds(K* kern, int bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename Tin, typename Tdo, int NP, int CT>
hipError_t launch_back(const DeltaBwdArgs& a, hipStream_t stream) {
    const DeltaArgs& f = a.f;
    const auto kern = &delta_back_kernel<Tin, Tdo, NP, CT>;
    constexpr int bytes = (int)sizeof(BackSmem<Tin, Tdo, NP, CT>);
    static_assert(bytes <= 160 * 1024, "LDS of a workgroup");
    const hipError_t e = lds(kern, bytes);
    if (e != hipSuccess) return e;
    const int npb = a.pad / (16 * CT);
    const int64_t units = (f.batch * f.H + 7) / 8 * 8;
    KTime kt("delta_back", stream);
    hipLaunchKernelGGL(kern, dim3((unsigned)(units * npb)), dim3(kBackThreads), bytes, stream, a, delta_chunks(f.L), npb);
    return hipGetLastError();
}

template <typename Tin, typename Tdo, int NP>
hipError_t launch(const DeltaBwdArgs& a, hipStream_t stream) {
    const DeltaArgs& f = a.f;
    const int64_t nch = delta_chunks(f.L);
    hipError_t e = launch_delta_prep(f, sizeof(Tin) == 2, true, a.recs, stream);
    if (e != hipSuccess) return e;
    e = launch_delta_keep(f, sizeof(Tin) == 2, a.recs, a.S, a.U, a.pad, stream);
    if (e != hipSuccess) return e;
    // Two column blocks to a workgroup where half as many still give each CU
    // one, as in the scan (batch 4, 16 heads of 128 x 128, L 2048: 146 us
    // against 194).  P of 16 and less too: the padded columns, which the
    // kernel after this one reads, cost a workgroup of their own otherwise
    // (batch 16, 32 heads of 16 x 64, L 1024: 141 us against 149).  float32
    // inputs: two blocks' LDS would not fit.
    bool two = false;
    if constexpr (sizeof(Tin) == 2) {
        two = f.batch * f.H * (a.pad / 32) >= host::device_cus();
        if (two) e = launch_back<Tin, Tdo, NP, 2>(a, stream);
    }
    if (!two) e = launch_back<Tin, Tdo, NP, 1>(a, stream);
    if (e != hipSuccess) return e;
    {
        const auto kern = &delta_grad_kernel<Tin, Tdo, NP>;
        constexpr int bytes = (int)sizeof(GradSmem<Tin, Tdo, NP>);
        static_assert(bytes <= 160 * 1024, "LDS of a workgroup");
        if ((e = lds(kern, bytes)) != hipSuccess) return e;
        KTime kt("delta_grad", stream);
        hipLaunchKernelGGL(kern, dim3((unsigned)(f.batch * f.H * nch)), dim3(kGradThreads), bytes, stream, a, nch);
    }
    if (a.pq) {
        KTime kt("delta_group", stream);
        const int64_t n = f.batch * f.L * f.G * f.N;
        hipLaunchKernelGGL((delta_group_kernel<Tin>), io::groups((n + 255) / 256), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

template <typename Tin, typename Tdo>
hipError_t by_n(const DeltaBwdArgs& a, hipStream_t stream) {
    return a.f.N <= 64 ? launch<Tin, Tdo, 64>(a, stream) : launch<Tin, Tdo, 128>(a, stream);
}

struct Sizes {
    size_t recs, state, rows, part;
};

Sizes sizes(int64_t batch, int64_t L, int64_t H, int64_t G, int64_t P, int64_t N) {
    const size_t chunks = (size_t)(batch * H * delta_chunks(L)), pad = (size_t)(P + 31) / 32 * 32;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    return {up(chunks * delta_record_bytes(true)), up(chunks * pad * (N <= 64 ? 64 : 128) * 4), up(chunks * kC * pad * 4),
            H > G ? up((size_t)(batch * L * H * N) * 4) : 0};
}

}  // namespace

size_t delta_bwd_bytes(int64_t batch, int64_t L, int64_t H, int64_t G, int64_t P, int64_t N) {
    const Sizes s = sizes(batch, L, H, G, P, N);
    return s.recs + 2 * s.state + 2 * s.rows + 2 * s.part;
}

void delta_bwd_carve(DeltaBwdArgs& a, void* ws) {
    const Sizes s = sizes(a.f.batch, a.f.L, a.f.H, a.f.G, a.f.P, a.f.N);
    char* p = static_cast<char*>(ws);
    auto take = [&](size_t n) {
        float* r = reinterpret_cast<float*>(p);
        p += n;
        return r;
    };
    a.recs = reinterpret_cast<char*>(take(s.recs));
    a.S = take(s.state);
    a.D = take(s.state);
    a.U = take(s.rows);
    a.dR = take(s.rows);
    a.pq = s.part ? take(s.part) : nullptr;
    a.pk = s.part ? take(s.part) : nullptr;
    a.pad = (int)((a.f.P + 31) / 32 * 32);
}

hipError_t launch_delta_bwd(const DeltaBwdArgs& a, int in_bf16, int out_bf16, hipStream_t stream) {
    if (in_bf16) return out_bf16 ? by_n<uint16_t, uint16_t>(a, stream) : by_n<uint16_t, float>(a, stream);
    return out_bf16 ? by_n<float, uint16_t>(a, stream) : by_n<float, float>(a, stream);
}

}  // namespace selscan
