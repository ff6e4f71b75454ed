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
// workgroup owns 16 or 32 columns of one head and walks its chunks in order.  The
// walk is a chain of three products a chunk, so what bounds it is their
// latency, and eight waves share each chunk.  Four state waves split the
// chain: wave w has the tokens 16 w .. 16 w + 15 of R and U and a quarter of
// the state's rows.  What a wave makes the others need as a B operand: split
// into planes it goes through LDS, three barriers a chunk.  Four helper
// waves, one beside each state wave on its SIMD, do what is not on the
// chain: Y (Q S while the state waves make U, A U a chunk later), staging K,
// needed both ways up, in LDS, and most of the loads, a chunk ahead.
//
// Measured: 16 heads of 128 x 128 (128 workgroups), L 16384, bf16: 419 us,
// 1.6 us a chunk (one wave to a column block: 1830 us; four that share its
// products: 730 us); 256 heads of 64 x 128, L 4096, fp32 y: 360 us, 0.95 GB of
// inputs, records and y (2.6 TB/s).  The matrix cores are busy for 11 and 28 %
// of it.  A chunk's 3850 cycles in the first: K S 1150 and 220 at the barrier, T R
// 730-1080 (by row block) and 200-600, K^T W 800 and 360.  T staged in LDS by
// the helpers was slower; a raised wave priority, and Q S, staging and A U one
// phase earlier, were no faster.
//
// Products are fp32-grade (split_mfma.hpp) whatever y's type: a bf16 y is the
// rounding of the fp32 one.
#include "delta_chunk.hpp"
#include "host.hpp"

namespace selscan {

namespace {

using namespace dchunk;

constexpr int kThreads = 512;

// KEEP: no y, and U has no second reader.
template <typename Tin, int NP, int CT, bool KEEP>
struct ScanSmem {
    static constexpr int kRow = NP + 8;
    float gam[kC], tail[kC], beta[kC];
    Tiles V[CT];
    uint16_t K[2][kPlanes<Tin>][kC][kRow];   // by chunk parity
    Operands<NP / 32, 3> S[CT];
    Operands<2, 3> R[CT], W[CT];             // R; e^(last - cum) U
    Operands<2, KEEP ? 1 : 3> U[CT];
};

// KEEP: instead of y, the state entering each chunk (kept_tile) and U
// [chunk, 64, pad], which the gradients read (pad: P rounded up to 32, the
// columns past P zero).  bf16 in and out with one column block, and KEEP: two
// workgroups to a CU (registers for four waves a SIMD), which such grids, up
// to twice the CUs, need to run at once.
template <typename Tin, typename Tout, int NP, int CT, bool KEEP>
__global__ __launch_bounds__(kThreads, CT == 1 && sizeof(Tin) == 2 && (KEEP || sizeof(Tout) == 2) ? 4 : 2)
void delta_scan_kernel(DeltaArgs a, const char* recs, int64_t nch, int npb, float* keep_s, float* keep_u, int pad) {
    constexpr int NK = kPlanes<Tin>, NU = KEEP ? 1 : 3;
    constexpr int ES = (int)sizeof(Tin), EO = (int)sizeof(Tout);
    constexpr int kRow = ScanSmem<Tin, NP, CT, KEEP>::kRow;
    constexpr int KS = NP / 32;              // k-steps over the key dimension
    constexpr int NT = NP / 64;              // state tiles per state wave
    constexpr int NPC = NP / 32;             // 8-element pieces of K per helper thread
    using Rc = Rec<KEEP>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<ScanSmem<Tin, NP, CT, KEEP>*>(smem_raw);
    const int tid = threadIdx.x & 255, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool helper = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0;
    // the column blocks of a head on one XCD (workgroups go round the eight),
    // whose L2 then serves its K, Q and records once from memory
    const int jx = blockIdx.x / 8;
    const int64_t bh = (int64_t)(jx / npb) * 8 + blockIdx.x % 8;
    if (bh >= a.batch * a.H) return;
    const int64_t b = bh / a.H, h = bh - b * a.H, grp = h / (a.H / a.G);
    const int64_t len = seq_len(a, b);
    const Chunks seq(len), all(a.L);         // of the sequence; of the tensors
    const int mine = seq.n;
    const int N = a.N, P = (int)a.P;
    const int p0 = (jx % npb) * 16 * CT + li;   // the lane's first column; the others 16 apart
    // strides of a token in bytes
    const int sk = scalar((int)(a.G * a.qk_row * ES)), sv = scalar((int)(a.H * P * ES)), sy = scalar((int)(a.H * P * EO));
    const int64_t krow = b * a.L * sk + grp * a.qk_row * ES;
    const char* Kg = scalar(static_cast<const char*>(a.k) + krow);
    const char* Qg = scalar(static_cast<const char*>(a.q) + krow);
    const char* Vg = scalar(static_cast<const char*>(a.v) + b * a.L * sv + h * P * ES);
    char* Yg = scalar(static_cast<char*>(a.y) + b * a.L * sy + h * P * EO);
    const char* Rg = scalar(recs + bh * nch * Rc::bytes);
    const f32x4 z4 = {0.0f, 0.0f, 0.0f, 0.0f};

    // Inputs are asked for as soon as the chunk before has used their
    // registers, a chunk's work ahead.  (Past the end: buffers of no rows.)
    // Loads and stores complete in order: stores go out after a phase's
    // loads, so that the waits for those find only stores a chunk older.
    auto chunk_rows = [&](const char* base, int stride, int c, int bytes) {
        return rows_buf(base + (int64_t)c * kC * stride, seq.rows(c), stride, bytes);
    };
    auto record = [&](int c) { return rows_buf(Rg + (int64_t)c * Rc::bytes, c < mine ? 1 : 0, 0, Rc::bytes); };
    int toff[2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) toff[ks] = row_of(w, ks, lane);

    if (!helper) {
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
        bf16x8 ft[2][3];
        auto fetch_t = [&](int c) {
            const auto rb = record(c);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int x = 0; x < 3; ++x) ft[ks][x] = buf_op(rb, toff[ks] + Rc::T + x * kPlane);
        };
        put_state();
        fetch_t(0);
        lds_barrier();
        for (int c = 0; c < mine; ++c) {
            const uint16_t* K = &sm.K[c & 1][0][0][0];
            // R for the wave's tokens
            f32x4 u[CT];
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
                }
            }
            auto gate = [&](const float* g) { return *reinterpret_cast<const f32x4*>(g + 16 * w + 4 * lg); };
            const f32x4 gam = gate(sm.gam), tail = gate(sm.tail), beta = gate(sm.beta);
            const float gl = sm.gam[kC - 1];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const f32x4 v = sm.V[ct].get(w, lane);
                f32x4 r;
#pragma unroll
                for (int q = 0; q < 4; ++q) r[q] = beta[q] * __builtin_fmaf(-gam[q], u[ct][q], v[q]);
                sm.R[ct].put_tile(w, r, lane);
                if constexpr (KEEP) {
                    float* ks = keep_s + (bh * nch + c) * pad * NP + kept_tile<NP>(p0 - li + 16 * ct, NT * w, lane);
#pragma unroll
                    for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4*>(ks + 256 * i) = S[i][ct];
                }
            }
            lds_barrier();
            // U for the wave's tokens (the first two waves' T ends in the first k-step)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bf16x8 x[2][3];
                sm.R[ct].get(0, lane, x[0]);
                if (w < 2) {
                    u[ct] = mm<3>(ft[0], x[0], z4);
                } else {
                    sm.R[ct].get(1, lane, x[1]);
                    u[ct] = mm_pair(ft, x);
                }
                sm.W[ct].put_tile(w, u[ct] * tail, lane);
                if constexpr (!KEEP) sm.U[ct].put_tile(w, u[ct], lane);
            }
            fetch_t(c + 1);
            bf16x8 k[NT * 2][NK];
            auto load_kt = [&]() {
#pragma unroll
                for (int i = 0; i < NT * 2; ++i)
#pragma unroll
                    for (int l = 0; l < NK; ++l)
                        k[i][l] = ld_down(K + l * kC * kRow, kRow, 32 * (i & 1), 16 * (NT * w + i / 2), lane);
            };
            // before the barrier that it does not need, where registers allow
            if constexpr (KEEP) load_kt();
            if constexpr (KEEP) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    float* ku = keep_u + (bh * nch + c) * kC * pad + p0 + 16 * ct;
#pragma unroll
                    for (int q = 0; q < 4; ++q) ku[(16 * w + 4 * lg + q) * pad] = u[ct][q];
                }
            }
            lds_barrier();
            // the wave's rows of the next state
            if constexpr (!KEEP) load_kt();
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
            put_state();
            lds_barrier();
        }
        if (!KEEP && a.last) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = 16 * (NT * w + i) + 4 * lg + q, p = p0 + 16 * ct;
                        if (p < P && n < N) a.last[(bh * P + p) * N + n] = S[i][ct][q];
                    }
        }
        return;
    }

    // ---- helper waves
    int koff[NPC], qoff[KS];
#pragma unroll
    for (int i = 0; i < NPC; ++i) {
        const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
        koff[i] = n0 < a.NL ? r * sk + n0 * ES : kOut;
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const int n = 32 * ks + 8 * lg;
        qoff[ks] = n < a.NL ? (16 * w + li) * sk + n * ES : kOut;
    }
    int yoff[CT], voff[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int p = p0 + 16 * ct;
        yoff[ct] = p < P ? (16 * w + 4 * lg) * sy + p * EO : kOut;
        voff[ct] = p < P ? (16 * w + 4 * lg) * sv + p * ES : kOut;
    }
    Raw8<Tin> fk[NPC], fq[KS];
    bf16x8 fa[2][NU];
    f32x4 fgam;
    auto fetch_k = [&](int c) {
        const auto kb = chunk_rows(Kg, sk, c, a.NL * ES);
#pragma unroll
        for (int i = 0; i < NPC; ++i) fetch8(kb, koff[i], fk[i]);
    };
    auto fetch_q = [&](int c) {
        const auto qb = chunk_rows(Qg, sk, c, a.NL * ES);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) fetch8(qb, qoff[ks], fq[ks]);
        fgam = buf_ld4(record(c), Rc::gam + (16 * w + 4 * lg) * 4);
    };
    auto fetch_a = [&](int c) {
        const auto rb = record(c);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int x = 0; x < NU; ++x) fa[ks][x] = buf_op(rb, toff[ks] + Rc::A + x * kPlane);
    };
    f32x4 fgate;
    Tin fv[CT][4];
    auto fetch_v = [&](int c) {
        const auto vb = chunk_rows(Vg, sv, c, P * ES);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int q = 0; q < 4; ++q) fv[ct][q] = buf_raw<Tin>(vb, voff[ct] + q * sv);
        fgate = buf_ld4(record(c), tid < 48 ? Rc::gam + 16 * tid : kOut);
    };
    auto stage_v = [&]() {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) sm.V[ct].put(w, widen(fv[ct]), lane);
        if (tid < 48) *reinterpret_cast<f32x4*>(&sm.gam[4 * tid]) = fgate;   // gam, tail, beta in a row
    };
    auto stage_k = [&](int c) {
#pragma unroll
        for (int i = 0; i < NPC; ++i) {
            const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            stage8(sm.K[c & 1][0][r], kC * kRow, n0, fk[i]);
        }
    };
    // Y of chunk c from y = e^cum Q S, its A in fa and its U in LDS
    auto finish_y = [&](int c, f32x4 (&y)[CT]) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            bf16x8 x[NU];
            sm.U[ct].get(0, lane, x);
            y[ct] = mm<3>(fa[0], x, y[ct]);
            if (w >= 2) {
                sm.U[ct].get(1, lane, x);
                y[ct] = mm<3>(fa[1], x, y[ct]);
            }
        }
        fetch_a(c + 1);
        const auto yb = rows_buf(Yg + (int64_t)c * kC * sy, all.rows(c), sy, P * EO);
        // (past the end a select: a row of zeros times a state that is not finite is not zero)
        const int live = seq.rows(c) - (16 * w + 4 * lg);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int q = 0; q < 4; ++q) buf_st(yb, yoff[ct] + q * sy, q < live ? a.scale * y[ct][q] : 0.0f, Tout(0));
    };
    fetch_k(0);
    fetch_v(0);
    if constexpr (!KEEP) {
        fetch_q(0);
        fetch_a(0);
    }
    stage_k(0);
    stage_v();
    fetch_k(1);
    fetch_v(1);
    f32x4 y[CT];
    lds_barrier();
    for (int c = 0; c < mine; ++c) {
        if constexpr (!KEEP) {
            if (c > 0) finish_y(c - 1, y);
        }
        lds_barrier();
        if constexpr (!KEEP) {
            constexpr int M = 2;   // k-steps at a time, as registers allow
            f32x4 acc[CT][M];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < M; ++i) acc[ct][i] = z4;
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += M) {
                bf16x8 x[M][NK];
#pragma unroll
                for (int i = 0; i < M; ++i) to_operand(fq[k0 + i], x[i]);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    bf16x8 s[M][3];
#pragma unroll
                    for (int i = 0; i < M; ++i) sm.S[ct].get(k0 + i, lane, s[i]);
                    mm_turns<3, NK, 3>([&](int m) { return x[m]; }, [&](int m) { return s[m]; }, acc[ct]);
                }
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) y[ct] = sum_of(acc[ct]) * fgam;
            fetch_q(c + 1);
        }
        lds_barrier();
        stage_k(c + 1);
        stage_v();
        fetch_k(c + 2);
        fetch_v(c + 2);
        lds_barrier();
    }
    if constexpr (!KEEP) {
        if (mine > 0) finish_y(mine - 1, y);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            if (p0 + 16 * ct < P)
                for (int64_t t = (int64_t)mine * kC + 4 * w + lg; t < a.L; t += 16)
                    io::st(reinterpret_cast<Tout*>(Yg + t * sy) + p0 + 16 * ct, 0.0f);
    }
}

template <typename Tin, typename Tout, int NP, int CT, bool KEEP>
hipError_t launch_ct(const DeltaArgs& a, const char* recs, float* keep_s, float* keep_u, int pad, hipStream_t stream) {
    constexpr int bytes = (int)sizeof(ScanSmem<Tin, NP, CT, KEEP>);
    static_assert(bytes <= 160 * 1024, "LDS of a workgroup");
    const int npb = (int)(((KEEP ? pad : a.P) + 16 * CT - 1) / (16 * CT));
    const int64_t units = (a.batch * a.H + 7) / 8 * 8;
    const auto kern = &delta_scan_kernel<Tin, Tout, NP, CT, KEEP>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    KTime kt(KEEP ? "delta_keep" : "delta_scan", stream);
    hipLaunchKernelGGL(kern, dim3((unsigned)(units * npb)), dim3(kThreads), bytes, stream, a, recs, delta_chunks(a.L), npb,
                       keep_s, keep_u, pad);
    return hipGetLastError();
}

template <typename Tin, typename Tout, int NP, bool KEEP>
hipError_t launch(const DeltaArgs& a, const char* recs, float* keep_s, float* keep_u, int pad, hipStream_t stream) {
    // Two column blocks to a workgroup share K's staging, its operands and
    // the barriers, but a chunk takes longer: worth it where half as many
    // workgroups still give each CU one (batch 8, 32 heads of 64 x 128, L
    // 4096, f32 y: 356 us against 486; the scan of the gradients at batch 4,
    // 16 heads of 128 x 128, L 2048: 92 against 105), not where CUs would
    // idle (batch 1, 16 heads of 128 x 128, L 16384: 614 us against 421).
    // float32 inputs: K's planes and two blocks do not fit a CU's LDS.
    if constexpr (sizeof(Tin) == 2) {
        const int64_t blocks = ((KEEP ? pad : a.P) + 31) / 32;
        if (a.P > 16 && a.batch * a.H * blocks >= host::device_cus())
            return launch_ct<Tin, Tout, NP, 2, KEEP>(a, recs, keep_s, keep_u, pad, stream);
    }
    return launch_ct<Tin, Tout, NP, 1, KEEP>(a, recs, keep_s, keep_u, pad, stream);
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
