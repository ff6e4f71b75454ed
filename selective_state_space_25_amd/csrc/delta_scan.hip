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
// S_t = e^g_t S_{t-1} + k_t u_t^T.  Value columns are independent: a
// workgroup owns 16 CT columns of one head and walks its chunks in order.
// The walk is a chain of three products a chunk, so what bounds it is their
// latency, and the four waves split each of them: wave w has the tokens
// 16 w .. 16 w + 15 of R, U and Y and a quarter of the state's rows.  What a
// wave makes the others need as a B operand, which a C tile pair is (see
// split_mfma.hpp): split into planes it goes through LDS, three barriers a
// chunk.  A wave's rows of Q, T and A are nobody else's and come from memory
// straight into its registers; only K, needed both ways up, is staged.  All
// of a chunk's inputs are fetched a chunk ahead.
//
// Products are fp32-grade (split_mfma.hpp) where they reach the state.  What
// goes into a bf16 y alone (Q S, A U) keeps plane pairs a + b < 2, an error
// near 2^-16 under the 2^-9 of y's own rounding.
#include <cstdlib>

#include "delta_chunk.hpp"

namespace selscan {

namespace {

using namespace dchunk;

// OL: plane pairs a + b < OL in the products of y; 0 = no y.
template <typename Tin, int NP, int CT, int OL>
struct ScanSmem {
    static constexpr int kRow = NP + 8;
    uint16_t K[2][kPlanes<Tin>][kC][kRow];   // by chunk parity
    Operands<NP / 32, 3> S[CT];
    Operands<2, 3> R[CT], W[CT];             // R; e^(last - cum) U
    Operands<2, OL ? OL : 1> U[CT];
};

// KEEP: instead of y, the state entering each chunk (kept_tile) and U
// [chunk, 64, pad], which the gradients read (pad: P rounded up to 32, the
// columns past P zero).
template <typename Tin, typename Tout, int NP, int CT, bool KEEP>
__global__ __launch_bounds__(256) void delta_scan_kernel(DeltaArgs a, const char* recs, int64_t nch, int npb,
                                                         float* keep_s, float* keep_u, int pad) {
    constexpr int OL = KEEP ? 0 : sizeof(Tout) == 2 ? 2 : 3;
    constexpr int OA = OL ? OL : 1;
    constexpr int NK = kPlanes<Tin>;
    constexpr int ES = (int)sizeof(Tin), EO = (int)sizeof(Tout);
    constexpr int kRow = ScanSmem<Tin, NP, CT, OL>::kRow;
    constexpr int KS = NP / 32;              // k-steps over the key dimension
    constexpr int NT = NP / 64;              // state tiles per wave
    constexpr int NPC = NP / 32;             // 8-element pieces of K per thread
    using R = Rec<KEEP ? 3 : OA, KEEP>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<ScanSmem<Tin, NP, CT, OL>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the column blocks of a head on one XCD (workgroups go round the eight),
    // whose L2 then serves its K, Q and records once from memory
    const int jx = blockIdx.x / 8;
    const int64_t bh = (int64_t)(jx / npb) * 8 + blockIdx.x % 8;
    if (bh >= a.batch * a.H) return;
    const int64_t b = bh / a.H, h = bh - b * a.H, grp = h / (a.H / a.G);
    const int64_t len = seq_len(a, b);
    const int mine = (int)((len + kC - 1) / kC);
    const int N = a.N, P = (int)a.P;
    const int p0 = (jx % npb) * 16 * CT + li;   // the lane's first column
    // strides of a token in bytes; chunk 0's rows
    const int64_t sk = a.G * a.qk_row * ES, sv = a.H * P * ES, sy = a.H * P * EO;
    const char* Kg = static_cast<const char*>(a.k) + b * a.L * sk + grp * a.qk_row * ES;
    const char* Qg = static_cast<const char*>(a.q) + b * a.L * sk + grp * a.qk_row * ES;
    const char* Vg = static_cast<const char*>(a.v) + b * a.L * sv + h * P * ES;
    char* Yg = static_cast<char*>(a.y) + b * a.L * sy + h * P * EO;

    f32x4 S[NT][CT];   // tile i: rows n = 16 (NT w + i) + 4 lg + q, column p0 + 16 ct
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = 16 * (NT * w + i) + 4 * lg + q, p = p0 + 16 * ct;
                S[i][ct][q] = a.h0 && p < P && n < N ? a.h0[(bh * P + p) * N + n] : 0.0f;
            }
    auto put_state = [&]() {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int i = 0; i < NT; ++i) sm.S[ct].put_tile(NT * w + i, S[i][ct], lane);
    };

    int koff[NPC], qoff[KS], toff[2], voff[CT], yoff[CT];
#pragma unroll
    for (int i = 0; i < NPC; ++i) {
        const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
        koff[i] = n0 < a.NL ? r * (int)sk + n0 * ES : kOut;
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int p = p0 + 16 * ct;
        voff[ct] = p < P ? (16 * w + 4 * lg) * (int)sv + p * ES : kOut;
        yoff[ct] = p < P ? (16 * w + 4 * lg) * (int)sy + p * EO : kOut;
    }

#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const int n = 32 * ks + 8 * lg;
        qoff[ks] = n < a.NL ? (16 * w + li) * (int)sk + n * ES : kOut;
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) toff[ks] = row_of(w, ks, lane);

    // A chunk's inputs on their way: each is asked for as soon as the chunk
    // before has used its registers, so that a whole chunk's work covers
    // memory's latency and no phase is held up issuing them all.  (Past the
    // end the last chunk is read again.)  Loads and stores complete in order:
    // y is stored after its phase's loads, so that the waits for those find
    // only stores a chunk older.
    Raw8<Tin> fk[NPC], fq[KS];
    bf16x8 ft[2][3], fa[2][OA];
    f32x4 fgate[3];
    float fgl;
    Tin fv[CT][4];
    auto rows = [&](const char* base, int64_t stride, int c, int bytes) {
        const int64_t t0 = (int64_t)min(c, mine - 1) * kC;
        return rows_buf(base + t0 * stride, (int)min((int64_t)kC, len - t0), stride, bytes);
    };
    auto record = [&](int c) { return rows_buf(recs + (bh * nch + min(c, mine - 1)) * R::bytes, 1, 0, R::bytes); };
    auto fetch_k = [&](int c) {
        const auto kb = rows(Kg, sk, c, a.NL * ES);
#pragma unroll
        for (int i = 0; i < NPC; ++i) fetch8(kb, koff[i], fk[i]);
    };
    auto fetch_q = [&](int c) {
        const auto qb = rows(Qg, sk, c, a.NL * ES);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) fetch8(qb, qoff[ks], fq[ks]);
    };
    auto fetch_v = [&](int c) {
        const auto vb = rows(Vg, sv, c, P * ES);
        const auto rb = record(c);
#pragma unroll
        for (int i = 0; i < 3; ++i) fgate[i] = buf_ld4(rb, R::gam + (i * kC + 16 * w + 4 * lg) * 4);
        fgl = buf_raw<float>(rb, R::gam + (kC - 1) * 4);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int q = 0; q < 4; ++q) fv[ct][q] = buf_raw<Tin>(vb, voff[ct] + q * (int)sv);
    };
    auto fetch_t = [&](int c) {
        const auto rb = record(c);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int x = 0; x < 3; ++x) ft[ks][x] = buf_op(rb, toff[ks] + R::T + x * kPlane);
    };
    auto fetch_a = [&](int c) {
        const auto rb = record(c);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int x = 0; x < OA; ++x) fa[ks][x] = buf_op(rb, toff[ks] + R::A + x * kPlane);
    };
    auto stage_k = [&](int c) {
#pragma unroll
        for (int i = 0; i < NPC; ++i) {
            const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            stage8(sm.K[c & 1][0][r], kC * kRow, n0, fk[i]);
        }
    };

    put_state();
    if (mine > 0) {
        fetch_k(0);
        fetch_v(0);
        fetch_t(0);
        if constexpr (!KEEP) {
            fetch_q(0);
            fetch_a(0);
        }
        stage_k(0);
        fetch_k(1);
    }
    lds_barrier();
    for (int c = 0; c < mine; ++c) {
        const int64_t t0 = (int64_t)c * kC;
        const uint16_t* K = &sm.K[c & 1][0][0][0];
        const f32x4 z4 = {0.0f, 0.0f, 0.0f, 0.0f};
        // R for the wave's tokens; Q S
        f32x4 y[CT], u[CT];
        {
            bf16x8 k[KS][NK];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int x = 0; x < NK; ++x) k[ks][x] = ld8(K + (x * kC + 16 * w + li) * kRow + 32 * ks + 8 * lg);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bf16x8 s[KS][3];
                f32x4 acc[KS];
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    sm.S[ct].get(ks, lane, s[ks]);
                    acc[ks] = z4;
                }
                mm_turns<3, NK, 3>([&](int m) { return k[m]; }, [&](int m) { return s[m]; }, acc);
                u[ct] = sum_of(acc);
                if constexpr (!KEEP) {
                    bf16x8 x[KS][NK];
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        to_operand(fq[ks], x[ks]);
                        acc[ks] = z4;
                    }
                    mm_turns<OA, NK, 3>([&](int m) { return x[m]; }, [&](int m) { return s[m]; }, acc);
                    y[ct] = sum_of(acc);
                }
            }
        }
        const f32x4 gam = fgate[0], tail = fgate[1], beta = fgate[2];
        const float gl = fgl;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const f32x4 v = widen(fv[ct]);
            f32x4 r;
#pragma unroll
            for (int q = 0; q < 4; ++q) r[q] = beta[q] * __builtin_fmaf(-gam[q], u[ct][q], v[q]);
            sm.R[ct].put_tile(w, r, lane);
        }
        fetch_v(c + 1);
        if constexpr (KEEP) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float* ks = keep_s + (bh * nch + c) * pad * NP + kept_tile<NP>(p0 - li + 16 * ct, NT * w, lane);
#pragma unroll
                for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4*>(ks + 256 * i) = S[i][ct];
            }
        }
        lds_barrier();
        // U for the wave's tokens (the first two waves' T ends in the first k-step)
        {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bf16x8 r[2][3];
                sm.R[ct].get(0, lane, r[0]);
                if (w < 2) {
                    u[ct] = mm<3>(ft[0], r[0], z4);
                } else {
                    sm.R[ct].get(1, lane, r[1]);
                    f32x4 acc[2] = {z4, z4};
                    mm_turns<3, 3, 3>([&](int m) { return ft[m]; }, [&](int m) { return r[m]; }, acc);
                    u[ct] = sum_of(acc);
                }
                sm.W[ct].put_tile(w, u[ct] * tail, lane);
                if constexpr (!KEEP) sm.U[ct].put_tile(w, u[ct], lane);
            }
        }
        fetch_t(c + 1);
        if constexpr (KEEP) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float* ku = keep_u + (bh * nch + c) * kC * pad + p0 + 16 * ct;
#pragma unroll
                for (int q = 0; q < 4; ++q) ku[(16 * w + 4 * lg + q) * pad] = u[ct][q];
            }
        } else {
            fetch_q(c + 1);
        }
        lds_barrier();
        // the wave's rows of the next state; Y
        {
            bf16x8 k[NT * 2][NK];
#pragma unroll
            for (int i = 0; i < NT * 2; ++i)
#pragma unroll
                for (int x = 0; x < NK; ++x)
                    k[i][x] = ld_down(K + x * kC * kRow, kRow, 32 * (i & 1), 16 * (NT * w + i / 2), lane);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bf16x8 x[2][3];
                sm.W[ct].get(0, lane, x[0]);
                sm.W[ct].get(1, lane, x[1]);
                f32x4 acc[NT * 2];
#pragma unroll
                for (int i = 0; i < NT * 2; ++i) acc[i] = i & 1 ? z4 : S[i / 2][ct] * gl;
                mm_turns<3, NK, 3>([&](int m) { return k[m]; }, [&](int m) { return x[m & 1]; }, acc);
#pragma unroll
                for (int i = 0; i < NT; ++i) S[i][ct] = acc[2 * i] + acc[2 * i + 1];
            }
        }
        put_state();
        stage_k(c + 1);
        fetch_k(c + 2);
        if constexpr (!KEEP) {
            const auto yb = rows_buf(Yg + t0 * sy, (int)min((int64_t)kC, a.L - t0), sy, P * EO);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bf16x8 x[2][OA];
                sm.U[ct].get(0, lane, x[0]);
                y[ct] *= gam;
                if (w < 2) {
                    y[ct] = mm<OA>(fa[0], x[0], y[ct]);
                } else {
                    sm.U[ct].get(1, lane, x[1]);
                    f32x4 acc[2] = {y[ct], z4};
                    mm_turns<OA, OA, OA>([&](int m) { return fa[m]; }, [&](int m) { return x[m]; }, acc);
                    y[ct] = sum_of(acc);
                }
            }
            fetch_a(c + 1);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
                for (int q = 0; q < 4; ++q) buf_st(yb, yoff[ct] + q * (int)sy, a.scale * y[ct][q], Tout(0));
            }
        }
        lds_barrier();
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int p = p0 + 16 * ct;
        if (p >= P) continue;
        if constexpr (!KEEP) {
            for (int64_t t = (int64_t)mine * kC + 4 * w + lg; t < a.L; t += 16)
                io::st(reinterpret_cast<Tout*>(Yg + t * sy) + p, 0.0f);
            if (a.last) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = 16 * (NT * w + i) + 4 * lg + q;
                        if (n < N) a.last[(bh * P + p) * N + n] = S[i][ct][q];
                    }
            }
        }
    }
}

// ------------------------------------------------ a wave per column block
// The same walk with the whole of a chunk's products of 16 columns in one
// wave: S, R and U never leave its registers (split_mfma.hpp's tile order),
// and the four waves of a workgroup, 64 columns, share K, Q, T and A in LDS.
template <typename Tin, int NP, int OL>
struct WideSmem {
    static constexpr int kRow = NP + 8;
    float gam[kC], tail[kC], beta[kC];
    uint16_t K[kPlanes<Tin>][kC][kRow];      // columns through kperm
    Frags<3, false> T;
    uint16_t Q[OL ? kPlanes<Tin> : 1][OL ? kC : 1][kRow];
    Frags<OL ? OL : 1, false> A;
};

template <typename Tin, typename Tout, int NP, bool KEEP>
__global__ __launch_bounds__(256) void delta_wide_kernel(DeltaArgs a, const char* recs, int64_t nch, int npb,
                                                         float* keep_s, float* keep_u, int pad) {
    constexpr int OL = KEEP ? 0 : sizeof(Tout) == 2 ? 2 : 3;
    constexpr int OA = OL ? OL : 1;
    constexpr int NK = kPlanes<Tin>;
    constexpr int ES = (int)sizeof(Tin), EO = (int)sizeof(Tout);
    using Smem = WideSmem<Tin, NP, OL>;
    constexpr int kRow = Smem::kRow;
    constexpr int NB = NP / 16, KS = NP / 32, NPC = NP / 32;
    using R = Rec<KEEP ? 3 : OA, KEEP>;
    constexpr int NM = (3 + (KEEP ? 0 : OL)) * kBlocks;     // 16 x 16 blocks in T's planes, and A's
    constexpr int NMT = (NM * 32 + 255) / 256;              // of which a thread takes so many half rows
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int jx = blockIdx.x / 8;
    const int64_t bh = (int64_t)(jx / npb) * 8 + blockIdx.x % 8;
    if (bh >= a.batch * a.H) return;
    const int64_t b = bh / a.H, h = bh - b * a.H, grp = h / (a.H / a.G);
    const int64_t len = seq_len(a, b);
    const int mine = (int)((len + kC - 1) / kC);
    const int N = a.N, P = (int)a.P;
    const int p = (jx % npb) * 64 + 16 * w + li;
    const bool active = p - li < (KEEP ? pad : P);
    const int64_t sk = a.G * a.qk_row * ES, sv = a.H * P * ES, sy = a.H * P * EO;
    const char* Kg = static_cast<const char*>(a.k) + b * a.L * sk + grp * a.qk_row * ES;
    const char* Qg = static_cast<const char*>(a.q) + b * a.L * sk + grp * a.qk_row * ES;
    const char* Vg = static_cast<const char*>(a.v) + b * a.L * sv + h * P * ES;
    char* Yg = static_cast<char*>(a.y) + b * a.L * sy + h * P * EO;

    f32x4 S[NB];   // tile i: rows n = 16 i + 4 lg + q, column p
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = 16 * i + 4 * lg + q;
            S[i][q] = a.h0 && p < P && n < N ? a.h0[(bh * P + p) * N + n] : 0.0f;
        }
    int koff[NPC], moff[NMT];
#pragma unroll
    for (int i = 0; i < NPC; ++i) {
        const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
        koff[i] = n0 < a.NL ? r * (int)sk + n0 * ES : kOut;
    }
#pragma unroll
    for (int i = 0; i < NMT; ++i) {
        const int id = tid + 256 * i;
        moff[i] = id < NM * 32 ? R::T + id * 16 : kOut;
    }
    const int voff = p < P ? 4 * lg * (int)sv + p * ES : kOut, yoff = p < P ? 4 * lg * (int)sy + p * EO : kOut;

    Raw8<Tin> fk[NPC], fq[NPC];
    u32x4 fm[NMT];
    f32x4 fgate;
    Tin fv[4][4];
    auto fetch = [&](int c) {
        const int64_t t0 = (int64_t)min(c, mine - 1) * kC;
        const int live = (int)min((int64_t)kC, len - t0);
        const auto kb = rows_buf(Kg + t0 * sk, live, sk, a.NL * ES);
        const auto qb = rows_buf(Qg + t0 * sk, live, sk, a.NL * ES);
        const auto vb = rows_buf(Vg + t0 * sv, live, sv, P * ES);
        const auto rb = rows_buf(recs + (bh * nch + t0 / kC) * R::bytes, 1, 0, R::bytes);
#pragma unroll
        for (int i = 0; i < NPC; ++i) {
            fetch8(kb, koff[i], fk[i]);
            if constexpr (!KEEP) fetch8(qb, koff[i], fq[i]);
        }
#pragma unroll
        for (int i = 0; i < NMT; ++i) fm[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, moff[i], 0, 0);
        fgate = buf_ld4(rb, tid < 48 ? R::gam + 16 * tid : kOut);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) fv[t][q] = buf_raw<Tin>(vb, voff + (16 * t + q) * (int)sv);
    };
    f32x4 v[4];
    auto stage = [&]() {
#pragma unroll
        for (int i = 0; i < NPC; ++i) {
            const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            stage8_perm(sm.K[0][r], kC * kRow, n0, fk[i]);
            if constexpr (!KEEP) stage8_perm(sm.Q[0][r], kC * kRow, n0, fq[i]);
        }
#pragma unroll
        for (int i = 0; i < NMT; ++i) {
            const int id = tid + 256 * i, blk = id >> 5, r = (id >> 1) & 15, c8 = id & 1;
            if (blk < 3 * kBlocks) sm.T.put(blk / kBlocks, blk % kBlocks, r, c8, fm[i]);
            else if (!KEEP && blk < NM) sm.A.put(blk / kBlocks - 3, blk % kBlocks, r, c8, fm[i]);
        }
        if (tid < 48) *reinterpret_cast<f32x4*>(&sm.gam[4 * tid]) = fgate;   // gam, tail, beta in a row
    };
    sm.T.clear(tid, 256);
    if constexpr (!KEEP) sm.A.clear(tid, 256);
    if (mine > 0) {
        fetch(0);
        stage();
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = widen(fv[t]);
    }
    lds_barrier();
    for (int c = 0; c < mine; ++c) {
        const int64_t t0 = (int64_t)c * kC;
        fetch(c + 1);
        if (active) {
            const f32x4 z4 = {0.0f, 0.0f, 0.0f, 0.0f};
            auto gate = [&](const float* g, int t) { return *reinterpret_cast<const f32x4*>(g + 16 * t + 4 * lg); };
            bf16x8 Sp[KS][3], Bp[2][3];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) split8<3>(S[2 * ks], S[2 * ks + 1], Sp[ks]);
            if constexpr (KEEP) {
                float* ks = keep_s + (bh * nch + c) * pad * NP + kept_tile<NP>(p - li, 0, lane);
#pragma unroll
                for (int i = 0; i < NB; ++i) *reinterpret_cast<f32x4*>(ks + 256 * i) = S[i];
            }
            f32x4 E[4], U[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) E[t] = U[t] = z4;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                bf16x8 k[4][NK];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int x = 0; x < NK; ++x) k[t][x] = ld8(&sm.K[x][16 * t + li][32 * ks + 8 * lg]);
                mm_turns<3, NK, 3>([&](int m) { return k[m]; }, [&](int) { return Sp[ks]; }, E);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4 gam = gate(sm.gam, t), beta = gate(sm.beta, t);
#pragma unroll
                for (int q = 0; q < 4; ++q) E[t][q] = beta[q] * __builtin_fmaf(-gam[q], E[t][q], v[t][q]);
            }
            split8<3>(E[0], E[1], Bp[0]);
            split8<3>(E[2], E[3], Bp[1]);
            {
                bf16x8 x[4][3];
#pragma unroll
                for (int t = 0; t < 4; ++t) sm.T.get(t, 0, lane, x[t]);
                mm_turns<3, 3, 3>([&](int m) { return x[m]; }, [&](int) { return Bp[0]; }, U);
                f32x4 u[2] = {z4, z4};
                sm.T.get(2, 1, lane, x[0]);
                sm.T.get(3, 1, lane, x[1]);
                mm_turns<3, 3, 3>([&](int m) { return x[m]; }, [&](int) { return Bp[1]; }, u);
                U[2] += u[0];
                U[3] += u[1];
            }
            if constexpr (KEEP) {
                float* ku = keep_u + ((bh * nch + c) * kC + 4 * lg) * pad + p;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) ku[(16 * t + q) * pad] = U[t][q];
            } else {
                bf16x8 Up[2][OA];
                split8<OA>(U[0], U[1], Up[0]);
                split8<OA>(U[2], U[3], Up[1]);
                const auto yb = rows_buf(Yg + t0 * sy, (int)min((int64_t)kC, a.L - t0), sy, P * EO);
                f32x4 y[4] = {z4, z4, z4, z4};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    bf16x8 x[4][NK];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int l = 0; l < NK; ++l) x[t][l] = ld8(&sm.Q[l][16 * t + li][32 * ks + 8 * lg]);
                    mm_turns<OA, NK, 3>([&](int m) { return x[m]; }, [&](int) { return Sp[ks]; }, y);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) y[t] *= gate(sm.gam, t);
                bf16x8 x[4][OA];
#pragma unroll
                for (int t = 0; t < 4; ++t) sm.A.get(t, 0, lane, x[t]);
                mm_turns<OA, OA, OA>([&](int m) { return x[m]; }, [&](int) { return Up[0]; }, y);
                f32x4 z[2] = {z4, z4};
                sm.A.get(2, 1, lane, x[0]);
                sm.A.get(3, 1, lane, x[1]);
                mm_turns<OA, OA, OA>([&](int m) { return x[m]; }, [&](int) { return Up[1]; }, z);
                y[2] += z[0];
                y[3] += z[1];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) buf_st(yb, yoff + (16 * t + q) * (int)sy, a.scale * y[t][q], Tout(0));
            }
            const float gl = sm.gam[kC - 1];
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] *= gate(sm.tail, t);
            split8<3>(U[0], U[1], Bp[0]);
            split8<3>(U[2], U[3], Bp[1]);
#pragma unroll
            for (int i = 0; i < NB; ++i) S[i] *= gl;
#pragma unroll
            for (int i = 0; i < NB; i += 4)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    bf16x8 k[4][NK];
                    f32x4 acc[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        acc[m] = S[i + m];
#pragma unroll
                        for (int x = 0; x < NK; ++x)
                            k[m][x] = ld_down_tile(&sm.K[x][0][0], kRow, 32 * ks, 16 * (i + m), lane);
                    }
                    mm_turns<3, NK, 3>([&](int m) { return k[m]; }, [&](int) { return Bp[ks]; }, acc);
#pragma unroll
                    for (int m = 0; m < 4; ++m) S[i + m] = acc[m];
                }
        }
        lds_barrier();
        stage();
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = widen(fv[t]);
        lds_barrier();
    }
    if (!KEEP && p < P) {
        for (int64_t t = (int64_t)mine * kC + lg; t < a.L; t += 4) io::st(reinterpret_cast<Tout*>(Yg + t * sy) + p, 0.0f);
        if (a.last) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = 16 * i + 4 * lg + q;
                    if (n < N) a.last[(bh * P + p) * N + n] = S[i][q];
                }
        }
    }
}

template <typename Tin, typename Tout, int NP, bool KEEP>
hipError_t launch(const DeltaArgs& a, const char* recs, float* keep_s, float* keep_u, int pad, hipStream_t stream) {
    constexpr int CT = 1;
    constexpr int OL = KEEP ? 0 : sizeof(Tout) == 2 ? 2 : 3;
    const int64_t units = (a.batch * a.H + 7) / 8 * 8;
    const bool wide = std::getenv("WIDE") != nullptr;
    const int cols = wide ? 64 : 16 * CT;
    const int npb = (int)(((KEEP ? pad : a.P) + cols - 1) / cols);
    const int bytes = wide ? (int)sizeof(WideSmem<Tin, NP, OL>) : (int)sizeof(ScanSmem<Tin, NP, CT, OL>);
    static_assert(sizeof(WideSmem<Tin, NP, OL>) <= 160 * 1024 && sizeof(ScanSmem<Tin, NP, CT, OL>) <= 160 * 1024,
                  "LDS of a workgroup");
    const auto kern = wide ? &delta_wide_kernel<Tin, Tout, NP, KEEP> : &delta_scan_kernel<Tin, Tout, NP, CT, KEEP>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    KTime kt(KEEP ? "delta_keep" : "delta_scan", stream);
    hipLaunchKernelGGL(kern, dim3((unsigned)(units * npb)), dim3(256), bytes, stream, a, recs, delta_chunks(a.L), npb,
                       keep_s, keep_u, pad);
    return hipGetLastError();
}

template <typename Tin, typename Tout>
hipError_t by_n(const DeltaArgs& a, const char* recs, hipStream_t stream) {
    return a.N <= 64 ? launch<Tin, Tout, 64, false>(a, recs, nullptr, nullptr, 0, stream)
                     : launch<Tin, Tout, 128, false>(a, recs, nullptr, nullptr, 0, stream);
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs& a, int in_bf16, int out_bf16, const char* recs, hipStream_t stream) {
    if (in_bf16) return out_bf16 ? by_n<uint16_t, uint16_t>(a, recs, stream) : by_n<uint16_t, float>(a, recs, stream);
    return out_bf16 ? by_n<float, uint16_t>(a, recs, stream) : by_n<float, float>(a, recs, stream);
}

hipError_t launch_delta_keep(const DeltaArgs& a, int in_bf16, const char* recs, float* keep_s, float* keep_u, int pad,
                             hipStream_t stream) {
    if (in_bf16) return a.N <= 64 ? launch<uint16_t, float, 64, true>(a, recs, keep_s, keep_u, pad, stream)
                                  : launch<uint16_t, float, 128, true>(a, recs, keep_s, keep_u, pad, stream);
    return a.N <= 64 ? launch<float, float, 64, true>(a, recs, keep_s, keep_u, pad, stream)
                     : launch<float, float, 128, true>(a, recs, keep_s, keep_u, pad, stream);
}

}  // namespace selscan
