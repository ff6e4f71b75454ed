// m2_chunk_scan.hip -- the Mamba-2 mixer's scan over 64-token chunks.
//
// With S [N, P] the state entering a chunk, cum_t the running sum of D_t A
// inside it, B, C and G = C B^T from m2_prep.hip and x = silu(conv), a head's
// outputs and next state are
//
//   Y  = e^cum (C S) + M X + D x,   M[t, s] = G[t, s] e^(cum_t - cum_s) D_s  (s <= t)
//   S' = e^last S + B^T (D e^(last - cum) X)
//
// and with X'_s = e^(r - cum_s) D_s x_s, r the middle of cum over the 32 tokens
// (0 and 1: the halves) that s is in,
//
//   M X = e^(cum - r0) (G X'0) + e^(cum - r1) (G X'1)
//   S'  = e^(last - r1) (e^(r1 - r0) (e^r0 S + B^T X'0) + B^T X'1)
//
// so that one split of X' into planes serves both products and G's planes are
// the group's, whatever the head.  Where the decays of 32 tokens span more than
// 2^120 the powers of two would leave fp32's range: such a chunk's M is made
// element by element.
//
// A wave owns 16 CT value columns of a head and walks the chunks with its S in
// accumulators, which are the operands of C S as they are: nothing of a head
// crosses waves.  The waves of a workgroup share a group's C, B and G, which
// go from memory into LDS without passing through registers, C while G X' and
// B^T X' run, B and G while C S runs: two barriers a chunk.  x is convolved by
// the lanes that multiply it, from the raw rows, and never written.
//
// A chunk's work does not depend on how many others are walked, so a sequence
// is cut into segments: a first pass makes each segment's state from zero
// (the B^T X' product alone), m2_carry_kernel joins them, and the second pass
// runs all segments at once from the states that enter them.  In a padded batch
// the device cuts the segments (m2_chunk.hpp), since the host does not know the
// lengths.
//
// 1 x 16384, 32 heads of 64 x 128 in one group, bf16, of a call of 220 us: 117
// us, 65 for the state pass, 17 for the carry between them and 21 for B and C
// (y in fp32: 120 of 225; fp32 inputs, one column block a wave: 138 of 242).
// Six MFMAs a product make this 0.17 TFLOP, 126 us of a library product's rate
// (1378 TFLOP/s), the state pass a fifth of it; the scan's matrix cores are busy
// 41 %, the vector ALU (convolution, splits, decays) 48 %, and a compute unit's
// one workgroup, two waves a SIMD, overlaps them as far as its two barriers a
// chunk let it.
//
// Products are fp32-grade (split_mfma.hpp).  cum is summed in fp64, and its
// exponentials take it as two fp32 parts: after strong decays it is large, and
// its rounding to one would be an error of them all.
#include <algorithm>

#include "host.hpp"
#include "lds_rows.hpp"
#include "m2_chunk.hpp"

namespace selscan {

namespace {

using namespace m2chunk;
using dchunk::buf_st;
using dchunk::kOut;
using dchunk::rows_buf;

// (lambdas that are called more than once would be calls, with a stack)
#define SELSCAN_INLINE __attribute__((always_inline))

constexpr int kWaves = 8;

// Most that the decays of 32 tokens span (log2) for r's powers of two: x D of
// 2^-30 keeps its three planes, of 2^60 stays finite.
constexpr double kSpan = 120.0;

// Per token of a wave's head: e^cum, e^(cum - r0), e^(cum - r1), D e^(r - cum).
// With decays past kSpan f0 and f1 are cum in two parts (log2), h is D.
struct Gates {
    float in[kC], f0[kC], f1[kC], h[kC];
};

template <int NP, int CT>
struct Smem {
    unsigned char C[Rec<NP>::blocks][kBlock];   // (the state pass: B of every other chunk)
    unsigned char B[Rec<NP>::blocks][kBlock];
    unsigned char G[18][kBlock];
    Gates gates[kWaves];
    float x[kWaves][CT][16][32];                // a k-step's x, a column a row (16-byte pieces exchanged by column)
};

// Sum over the lanes up to this one, by data-parallel moves (a lane that has
// none to take from adds zero).
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_moved(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, true);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum_to_lane(double v) {
    v = add_moved<0x111, 0xf>(v);   // 1, 2, 4, 8 lanes up within 16
    v = add_moved<0x112, 0xf>(v);
    v = add_moved<0x114, 0xf>(v);
    v = add_moved<0x118, 0xf>(v);
    v = add_moved<0x142, 0xa>(v);   // lane 15 to the second 16, 47 to the fourth
    return add_moved<0x143, 0xc>(v);   // lane 31 to the upper half
}
template <int LANE>
__device__ __forceinline__ double of_lane(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, LANE), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), LANE);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ float exp2_of(double d) {
    const float hi = (float)d, e = fast_exp2(hi);
    return __builtin_fmaf(e, (float)(d - (double)hi) * kLn2, e);
}

__device__ __forceinline__ uint32_t lds_at(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// CT neighbouring elements as loaded.
template <typename T, int CT> struct RawOf;
template <> struct RawOf<uint16_t, 1> { typedef uint16_t type; };
template <> struct RawOf<uint16_t, 2> { typedef uint32_t type; };
template <> struct RawOf<float, 1> { typedef float type; };
template <> struct RawOf<float, 2> { typedef float type __attribute__((ext_vector_type(2))); };
template <typename T, int CT> using RawX = typename RawOf<T, CT>::type;

template <typename T, int CT>
__device__ __forceinline__ RawX<T, CT> buf_x(__amdgpu_buffer_rsrc_t r, int off) {
    using RX = RawX<T, CT>;
    if constexpr (CT * sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    else if constexpr (CT * sizeof(T) == 4) return __builtin_bit_cast(RX, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    else return __builtin_bit_cast(RX, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
}
__device__ __forceinline__ void widen(uint16_t r, float (&v)[1]) { v[0] = bf16_to_f32(r); }
__device__ __forceinline__ void widen(uint32_t r, float (&v)[2]) { v[0] = bf16lo(r); v[1] = bf16hi(r); }
__device__ __forceinline__ void widen(float r, float (&v)[1]) { v[0] = r; }
__device__ __forceinline__ void widen(RawX<float, 2> r, float (&v)[2]) { v[0] = r[0]; v[1] = r[1]; }

// CT neighbouring results.
template <int CT, typename T>
__device__ __forceinline__ void store_y(__amdgpu_buffer_rsrc_t r, int off, const float (&v)[CT], T) {
    if constexpr (CT == 1) {
        buf_st(r, off, v[0], T(0));
    } else if constexpr (sizeof(T) == 2) {
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16x2(v[0], v[1]), r, off, 0, 0);
    } else {
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(v[0]), __float_as_uint(v[1])}, r, off, 0, 0);
    }
}

// `n` blocks from global memory into LDS, shared out over the workgroup's waves.
__device__ __forceinline__ void copy_blocks(const char* from, const void* to, int n, int wave, int waves, int lane) {
    const uint32_t slot = lds_at(to);
    for (int i = wave; i < n; i += waves) rows::dma_at<0>(from + i * kBlock + lane * 16, __builtin_amdgcn_readfirstlane(slot + i * kBlock));
}

// Everything that this wave asked of memory is there, and the other waves' too.
__device__ __forceinline__ void all_there() {
    rows::wait_vm();
    lds_barrier();
}

__device__ __forceinline__ bf16x8 op_at(const unsigned char (*blocks)[kBlock], int i, int lane) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(&blocks[i][lane * 16]));
}

// M products over one k-step, in turns: an MFMA that adds to the sum of the one
// before waits out its latency, and the compiler, which may move anything else
// between them, is kept from lining such up.
template <int M, typename FA, typename FB, typename FC>
__device__ __forceinline__ void in_turns(FA a, FB b, FC c) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i) {
#pragma unroll
            for (int m = 0; m < M; ++m) c(m) = mfma(a(m)[i], b(m)[s - i], c(m));
            __builtin_amdgcn_sched_barrier(0x496);   // (vector, scalar, memory and LDS instructions may pass)
        }
}

// STATE: the first pass, a segment's state from zero and the sum of its log2 decays.
template <typename Tin, typename Tout, int K, int NP, int CT, bool STATE>
__global__ __launch_bounds__(64 * kWaves, 2) void m2_chunk_kernel(M2ConvArgs a, Plan pl, const char* recs, float* seg_state,
                                                                 float* seg_log) {
    constexpr int KS = NP / 32, NT = NP / 16, ES = (int)sizeof(Tin), EO = (int)sizeof(Tout);
    using R = Rec<NP>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<Smem<NP, CT>*>(smem_raw);
    int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
    // Anew for each chunk: whatever follows from the lane alone would be kept in
    // registers throughout, and there are none left for it.
    auto place = [&]() SELSCAN_INLINE {
        lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        li = lane & 15;
        lg = lane >> 4;
    };
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the workgroups that share a segment's records on one XCD (workgroups go round the eight)
    const int64_t id = io::group_id(), oct = id / (8 * pl.sets), in8 = id - oct * 8 * pl.sets;
    const int64_t seg_id = oct * 8 + in8 % 8;
    const int set = (int)(in8 / 8);
    const int64_t bs = seg_id / a.G, grp = seg_id - bs * a.G;
    if (bs >= pl.all) return;
    int64_t b, seg, per;
    if (pl.segs) {
        b = bs / pl.segs;
        seg = bs - b * pl.segs;
        per = pl.per;
    } else {
        const Cut cut(a, pl);
        const int of = __popcll(__ballot(cut.n > 0 && cut.first <= bs)) - 1;
        b = of;
        seg = bs - __builtin_amdgcn_readlane(cut.first, of);
        per = scalar(cut.per);
        if (seg >= __builtin_amdgcn_readlane(cut.n, of)) return;
    }
    const int64_t len = seq_len(a, b);
    const int64_t nch = (len + kC - 1) / kC;
    const int64_t c0 = seg * per, c1 = min(c0 + per, nch);
    if (STATE && c1 >= nch) return;   // nothing follows this segment
    const int unit = set * pl.waves + wave;
    const bool live = unit < pl.units;
    const int64_t h = grp * (a.H / a.G) + (live ? unit / pl.cols : 0);
    const int p0 = (live ? unit % pl.cols : 0) * 16 * CT;   // the wave's first column; lane li has CT li and the one behind it
    const bool mine = live && p0 + CT * li < a.P;           // (CT = 2: P is even)
    Tout* Y = static_cast<Tout*>(a.y) + (b * a.L * a.H + h) * a.P;
    const int64_t yrow = a.H * a.P;
    if (c0 >= nch && c0 > 0) return;   // past the end
    Gates& gt = sm.gates[wave];
    const Tin* T = static_cast<const Tin*>(a.dt) + b * a.dt_batch + h;
    const float A = a.A[h], dt_bias = a.dt_bias ? a.dt_bias[h] : 0.0f, skip = a.D ? a.D[h] : 0.0f;
    const int64_t ch = h * a.P + p0 + CT * li, C = a.conv.C;
    const char* X0 = scalar(reinterpret_cast<const char*>(static_cast<const Tin*>(a.conv.x) + b * a.conv.x_batch + h * a.P));
    const Tin* XS = scalar(a.conv.state ? static_cast<const Tin*>(a.conv.state) + b * (K - 1) * C + h * a.P : nullptr);
    float w[K][CT], bias[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        bias[i] = mine && a.conv.bias ? a.conv.bias[ch + i] : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][i] = mine ? a.conv.weight[(ch + i) * K + k] : 0.0f;
    }
    // state tile nt: rows n = 16 nt + 4 lg + q, column p0 + ct
    f32x4 S[NT][CT];
    const int64_t srow = (b * a.H + h) * a.P + p0 + CT * li;
    const float* S0 = STATE ? nullptr
                      : c0 > 0  ? seg_state + (((seg_id / a.G) * a.H + h) * a.P + p0 + CT * li) * a.N
                      : a.h0    ? a.h0 + srow * a.N
                                : nullptr;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            S[i][ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            const int n = 16 * i + 4 * lg;
            if (S0 && mine && n < a.N) {
                io::Piece<float, 4> r;
                r.get(S0 + ct * a.N + n);
                S[i][ct] = r.v;
            }
        }
    char* Y0 = scalar(reinterpret_cast<char*>(Y));
    const char* rec0 = recs + (b * pl.chunks * a.G + grp) * R::bytes;
    const int64_t rec_row = a.G * R::bytes;
    auto fetch_dt = [&](int64_t c) SELSCAN_INLINE {
        const int64_t t = c * kC + lane;
        return t < len ? io::ld(T + t * a.dt_row) : 0.0f;
    };
    // The lane's raw x of a k-step: tokens 32 ks + 8 lg - (K - 1) .. + 7 of its
    // columns.  Past the end the buffer gives zero.
    using RX = RawX<Tin, CT>;
    RX xr[K - 1 + 8];
    const int xrow = scalar((int)(a.conv.x_row * ES)), xbytes = scalar((int)(a.P * ES));
    auto fetch_x = [&](int64_t c, int ks, bool later = true) SELSCAN_INLINE {   // later: chunk 0 it is not
        const int64_t t0 = c * kC;
        const int before = later ? K - 1 : 0;
        const auto xb = rows_buf(X0 + (t0 - before) * xrow, scalar((int)min((int64_t)(kC + before), len - t0 + before)), xrow, xbytes);
        const int at = mine ? (p0 + CT * li) * ES + (8 * lg + before - (K - 1)) * xrow : kOut;
#pragma unroll
        for (int j = 0; j < K - 1 + 8; ++j) xr[j] = buf_x<Tin, CT>(xb, at + (32 * ks + j) * xrow);
        if (!later && ks == 0 && lg == 0) {   // (rows that overlap reach back into the buffer, so not left to it)
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                io::Piece<Tin, CT> r;
                r.zero();
                if (XS && mine) r.get(XS + j * C + p0 + CT * li);
                xr[j] = __builtin_bit_cast(RX, r);
            }
        }
    };
    auto convolve = [&](int64_t c, int ks, float (&x)[CT][8]) {
        float r[K - 1 + 8][CT];
#pragma unroll
        for (int j = 0; j < K - 1 + 8; ++j) widen(xr[j], r[j]);
        const int in = scalar((int)min((int64_t)kC, len - c * kC)) - (32 * ks + 8 * lg);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                float pre = bias[i];
#pragma unroll
                for (int k = 0; k < K; ++k) pre = __builtin_fmaf(w[k][i], r[j + k][i], pre);
                x[i][j] = j < in ? silu_scaled(pre, 1.0f) : 0.0f;
            }
    };
    float dtv = c0 < c1 ? fetch_dt(c0) : 0.0f;
    double chunk_log = 0.0;   // its log2 decay
    // e^r0, e^(r1 - r0), e^(last - r1); past kSpan e^last, 1, 1, and last
    float front = 1.0f, mid = 1.0f, tail = 1.0f, last_hi = 0.0f, last_lo = 0.0f;
    bool narrow = true;   // the chunk's decays are within kSpan
    // the chunk's gates, a token a lane
    auto make_gates = [&](int64_t c) SELSCAN_INLINE {
        const bool in = c * kC + lane < len;
        const float sp = in ? softplus_log2((dtv + dt_bias) * kLog2e) : 0.0f;
        double cum = in ? (double)sp * (double)A : 0.0;
        cum = sum_to_lane(cum < -1e6 ? -1e6 : cum);   // (a decay of zero either way; stays finite)
        const double half = of_lane<31>(cum), last = of_lane<63>(cum);
        const double r0 = 0.5 * half, r1 = 0.5 * (half + last), r = lane < 32 ? r0 : r1;
        const float step = sp * kLn2;
        narrow = half >= -kSpan && last - half >= -kSpan && half <= 100.0 && last <= 100.0;
        if constexpr (!STATE) gt.in[lane] = exp2_of(cum);
        if (narrow) {
            if constexpr (!STATE) {
                gt.f0[lane] = exp2_of(cum - r0);
                gt.f1[lane] = exp2_of(cum - r1);
            }
            gt.h[lane] = step * exp2_of(r - cum);
        } else {
            const float hi = (float)cum;
            gt.f0[lane] = hi;
            gt.f1[lane] = (float)(cum - (double)hi);
            gt.h[lane] = step;
            last_hi = (float)last;
            last_lo = (float)(last - (double)last_hi);
        }
        front = exp2_of(narrow ? r0 : last);
        mid = exp2_of(narrow ? r1 - r0 : 0.0);
        tail = exp2_of(narrow ? last - r1 : 0.0);
        chunk_log = last;
        dchunk::wave_sync();
    };
    // X' of a k-step from its x
    auto scaled = [&](int ks, const float (&x)[CT][8], bf16x8 (&xp)[CT][3]) {
        const f32x4 h0 = *reinterpret_cast<const f32x4*>(&gt.h[32 * ks + 8 * lg]);
        const f32x4 h1 = *reinterpret_cast<const f32x4*>(&gt.h[32 * ks + 8 * lg + 4]);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            split8<3>(f32x4{x[ct][0], x[ct][1], x[ct][2], x[ct][3]} * h0, f32x4{x[ct][4], x[ct][5], x[ct][6], x[ct][7]} * h1, xp[ct]);
    };
    // what decays past kSpan leave to do: the values of planes times e^(to - cum_s), s = the k-step's tokens up to `most`
    auto decayed = [&](int ks, bf16x8 (&p)[3], float to_hi, float to_lo, int most) {
        const int s0 = 32 * ks + 8 * lg;
        asm volatile("" ::: "memory");   // (cum is read again each time: it has no registers to stay in)
        f32x4 v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const f32x4 hs = *reinterpret_cast<const f32x4*>(&gt.f0[s0 + 4 * e]);
            const f32x4 ls = *reinterpret_cast<const f32x4*>(&gt.f1[s0 + 4 * e]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float g = ((float)p[0][4 * e + j] + (float)p[1][4 * e + j]) + (float)p[2][4 * e + j];
                const float d = (to_hi - hs[j]) + (to_lo - ls[j]);
                v[e][j] = g * fast_exp2(s0 + 4 * e + j <= most ? d : -1e30f);   // (G above its diagonal is zero, not e^d)
            }
        }
        split8<3>(v[0], v[1], p);
    };
    auto decayed_x = [&](int ks, bf16x8 (&xp)[CT][3]) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) decayed(ks, xp[ct], last_hi, last_lo, kC);
    };
    auto scale_state = [&](float by) SELSCAN_INLINE {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) S[i][ct] *= by;
    };
    // S += B^T X' over a k-step
    auto write = [&](const unsigned char (*Bs)[kBlock], int ks, const bf16x8 (&xp)[CT][3]) {
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
            bf16x8 bp[2][3];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int x3 = 0; x3 < 3; ++x3) bp[k][x3] = op_at(Bs, ((i + k) * 2 + ks) * 3 + x3, lane);
            in_turns<2 * CT>([&](int m) -> const bf16x8(&)[3] { return bp[m / CT]; },
                             [&](int m) -> const bf16x8(&)[3] { return xp[m % CT]; },
                             [&](int m) -> f32x4& { return S[i + m / CT][m % CT]; });
        }
    };
    // A chunk's gates and its first raw x stand ready when it begins (the state
    // pass: its first X'), made beside the chunk before's last products.
    bf16x8 x0p[CT][3], x1p[CT][3];
    float x[CT][8];
    if (c0 < c1) {
        if (live) fetch_x(c0, 0, c0 > 0);
        make_gates(c0);
        if (STATE && live) {
            convolve(c0, 0, x);
            fetch_x(c0, 1, c0 > 0);
            scaled(0, x, x0p);
        }
        dtv = c0 + 1 < c1 ? fetch_dt(c0 + 1) : 0.0f;
    }
    if constexpr (STATE) {
        copy_blocks(rec0 + c0 * rec_row + R::B, sm.C, R::blocks, wave, pl.waves, lane);
        double seg_sum = 0.0;
        for (int64_t c = c0; c < c1; ++c) {
            place();
            seg_sum += chunk_log;
            all_there();
            const bool odd = (c - c0) & 1;
            const unsigned char(*Bs)[kBlock] = odd ? sm.B : sm.C;
            if (c + 1 < c1) copy_blocks(rec0 + (c + 1) * rec_row + R::B, odd ? sm.C : sm.B, R::blocks, wave, pl.waves, lane);
            if (live && !narrow) decayed_x(0, x0p);
            scale_state(front);
            if (live) {
                convolve(c, 1, x);
                fetch_x(c + 1, 0);
                scaled(1, x, x1p);
                write(Bs, 0, x0p);
                if (!narrow) decayed_x(1, x1p);
                scale_state(mid);
            }
            const float out = tail;
            make_gates(c + 1);
            if (live) {
                convolve(c + 1, 0, x);
                fetch_x(c + 1, 1);
                scaled(0, x, x0p);
                write(Bs, 1, x1p);
                scale_state(out);
            }
            dtv = c + 2 < c1 ? fetch_dt(c + 2) : 0.0f;
        }
        if (lane == 0 && live && unit % pl.cols == 0) seg_log[(seg_id / a.G) * a.H + h] = (float)seg_sum;
    } else {
        if (c0 < c1) copy_blocks(rec0 + c0 * rec_row + R::C, sm.C, R::blocks, wave, pl.waves, lane);
        float(&xs)[CT][16][32] = sm.x[wave];
        // a k-step's x into the order of y
        auto turn = [&]() SELSCAN_INLINE {
            dchunk::wave_sync();
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<f32x4*>(&xs[ct][li][4 * ((2 * lg + e) ^ (li & 7))]) =
                        f32x4{x[ct][4 * e], x[ct][4 * e + 1], x[ct][4 * e + 2], x[ct][4 * e + 3]};
            dchunk::wave_sync();
        };
        for (int64_t c = c0; c < c1; ++c) {
            const char* rec = rec0 + c * rec_row;
            place();
            all_there();   // C; and every wave is done with the chunk before
            copy_blocks(rec + R::B, sm.B, R::blocks + 18, wave, pl.waves, lane);   // and G, behind B in both
            f32x4 y[4][CT];
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) y[tt][ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (live) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    bf16x8 sp[CT][3];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) split8<3>(S[2 * ks][ct], S[2 * ks + 1][ct], sp[ct]);
#pragma unroll
                    for (int tt = 0; tt < 4; tt += 2) {
                        bf16x8 cp[2][3];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int x3 = 0; x3 < 3; ++x3) cp[k][x3] = op_at(sm.C, (ks * 4 + tt + k) * 3 + x3, lane);
                        in_turns<2 * CT>([&](int m) -> const bf16x8(&)[3] { return cp[m / CT]; },
                                         [&](int m) -> const bf16x8(&)[3] { return sp[m % CT]; },
                                         [&](int m) -> f32x4& { return y[tt + m / CT][m % CT]; });
                    }
                }
            }
            all_there();   // B and G; and every wave is done with C
            if (c + 1 < c1) copy_blocks(rec + rec_row + R::C, sm.C, R::blocks, wave, pl.waves, lane);
            if (!live) continue;
            const auto yb = rows_buf(Y0 + c * kC * yrow * EO, scalar((int)min((int64_t)kC, a.L - c * kC)), scalar((int)(yrow * EO)), scalar((int)(a.P * EO)));
            const int in = scalar((int)min((int64_t)kC, len - c * kC)) - 4 * lg;
            const int y0 = (mine ? (p0 + CT * li) * EO : kOut) + 4 * lg * (int)(yrow * EO);
            // G X' of a k-step; with decays past kSpan M X
            auto add_gx = [&](auto fast, int ks, const bf16x8 (&xp)[CT][3]) {
#pragma unroll
                for (int tt = 2 * ks; tt < 4; tt += 2) {
                    bf16x8 gp[2][3];
                    f32x4 acc[2][CT];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
#pragma unroll
                        for (int x3 = 0; x3 < 3; ++x3) gp[k][x3] = op_at(sm.G, g_tile(tt + k, ks) * 3 + x3, lane);
                        const int t = 16 * (tt + k) + li;
                        if constexpr (!decltype(fast)::value) decayed(ks, gp[k], gt.f0[t], gt.f1[t], t);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) acc[k][ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                    in_turns<2 * CT>([&](int m) -> const bf16x8(&)[3] { return gp[m / CT]; },
                                     [&](int m) -> const bf16x8(&)[3] { return xp[m % CT]; },
                                     [&](int m) -> f32x4& { return acc[m / CT][m % CT]; });
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        f32x4 f = {1.0f, 1.0f, 1.0f, 1.0f}, e = f;
                        if constexpr (decltype(fast)::value) f = *reinterpret_cast<const f32x4*>(&(ks ? gt.f1 : gt.f0)[16 * (tt + k) + 4 * lg]);
                        if (ks == 0) e = *reinterpret_cast<const f32x4*>(&gt.in[16 * (tt + k) + 4 * lg]);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) {
                            f32x4& v = y[tt + k][ct];
                            v = ks == 0 ? v * e + acc[k][ct] * f : v + acc[k][ct] * f;
                        }
                    }
                }
            };
            // the rows of a k-step's tokens
            auto put_y = [&](int ks) SELSCAN_INLINE {
#pragma unroll
                for (int tt = 2 * ks; tt < 2 * ks + 2; ++tt) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        y[tt][ct] += *reinterpret_cast<const f32x4*>(&xs[ct][li][4 * ((4 * (tt & 1) + lg) ^ (li & 7))]) * skip;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float v[CT];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) v[ct] = 16 * tt + q < in ? y[tt][ct][q] : 0.0f;
                        store_y<CT>(yb, y0 + (16 * tt + q) * (int)(yrow * EO), v, Tout(0));
                    }
                }
            };
            convolve(c, 0, x);
            fetch_x(c, 1, c > 0);
            turn();
            scaled(0, x, x0p);
            if (narrow) {
                add_gx(std::true_type(), 0, x0p);
            } else {
                add_gx(std::false_type(), 0, x0p);
                decayed_x(0, x0p);
            }
            put_y(0);
            scale_state(front);
            convolve(c, 1, x);
            fetch_x(c + 1, 0);
            scaled(1, x, x1p);
            write(sm.B, 0, x0p);
            turn();
            if (narrow) {
                add_gx(std::true_type(), 1, x1p);
            } else {
                add_gx(std::false_type(), 1, x1p);
                decayed_x(1, x1p);
            }
            put_y(1);
            scale_state(mid);
            const float out = tail;
            make_gates(c + 1);
            write(sm.B, 1, x1p);
            scale_state(out);
            dtv = c + 2 < c1 ? fetch_dt(c + 2) : 0.0f;
        }
        if (c1 < nch || !a.last) return;
    }
    float* S1 = STATE ? seg_state + (((seg_id / a.G + 1) * a.H + h) * a.P + p0 + CT * li) * a.N : a.last + srow * a.N;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const int n = 16 * i + 4 * lg;
            if (mine && n < a.N) {
                io::Piece<float, 4> r;
                r.v = S[i][ct];
                r.put(S1 + ct * a.N + n);
            }
        }
}

// The states that enter segments 1, 2, ..: slot s of seg_state holds what
// segment s - 1 made from zero, and takes the state entering segment s.  Four
// elements a thread.
__global__ __launch_bounds__(256) void m2_carry_kernel(M2ConvArgs a, Plan pl, float* seg_state, const float* seg_log) {
    const int64_t head = a.P * a.N, i = (io::group_id() * 256 + threadIdx.x) * 4;
    const int64_t bh = i / head, e = i - bh * head, b = bh / a.H, h = bh - b * a.H;
    int cut_n = 0, cut_first = 0;
    if (!pl.segs) {   // (all lanes)
        const Cut cut(a, pl);
        cut_n = __shfl(cut.n, (int)b & 63, 64);
        cut_first = __shfl(cut.first, (int)b & 63, 64);
    }
    if (b >= a.batch) return;
    const int64_t len = a.conv.lengths ? min((int64_t)max(a.conv.lengths[b], 0), a.L) : a.L;
    const int64_t n = pl.segs ? ((len + kC - 1) / kC + pl.per - 1) / pl.per : cut_n;   // the sequence's segments
    const int64_t s0 = pl.segs ? b * pl.segs : cut_first;
    io::Piece<float, 4> first;
    first.zero();
    if (a.h0) first.get(a.h0 + i);
    f32x4 s = first.v;
    constexpr int kAhead = 8;   // loads in flight
    for (int64_t g = 0; g + 1 < n; g += kAhead) {
        f32x4 u[kAhead];
        float d[kAhead];
        float* to = seg_state + ((s0 + g + 1) * a.H + h) * head + e;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (g + k + 1 < n) {
                u[k] = *reinterpret_cast<const f32x4*>(to + k * a.H * head);
                d[k] = fast_exp2(seg_log[(s0 + g + k) * a.H + h]);
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (g + k + 1 < n) *reinterpret_cast<f32x4*>(to + k * a.H * head) = s = s * d[k] + u[k];
    }
}

Plan plan_of(const M2ConvArgs& a, int in_bf16, bool ragged) {
    Plan p;
    p.chunks = (a.L + kC - 1) / kC;
    p.np = a.N <= 32 ? 32 : (int)a.N;
    const int64_t heads = a.H / a.G;
    // two column blocks a wave halve the reads of B and C from LDS; one where
    // a group would not fill a workgroup's waves, pairs of columns P, or (fp32,
    // N = 128) two blocks a wave's registers (1 x 16384 as above: 219 us a call
    // with two, 234 with one; 8 x 4096 ragged 268 and 309)
    p.ct = a.P % 2 || heads * ((a.P + 31) / 32) < kWaves || (!in_bf16 && p.np == 128) ? 1 : 2;
    p.cols = (int)((a.P + 16 * p.ct - 1) / (16 * p.ct));
    p.units = (int)(heads * p.cols);
    p.sets = (p.units + kWaves - 1) / kWaves;
    p.waves = (p.units + p.sets - 1) / p.sets;
    // Segments of two chunks and more: a workgroup for each compute unit, which
    // holds one (batch 1, L 16384, 32 heads of 64 x 128: 219 us, with two
    // workgroups a unit 247; 8 x 4096: 379 and 411).  Where sequences may end early and the shortest
    // segments would be more than that, the device cuts them from the tokens
    // that are there, four a sequence at least, in whole rounds of workgroups
    // (batch 8, lengths spread over 0 .. 4096: 268 us; segments of one length,
    // four workgroups a unit, 337).  Its cut costs 0.5 us a launch (batch 3 of
    // up to 333 tokens: 38 us, without 35), and a lane a sequence does no more
    // than 64: those have one length, and four workgroups a unit.
    const int64_t cus = host::device_cus(), groups = a.batch * a.G * p.sets;
    p.want = std::max<int64_t>(1, cus / (a.G * p.sets));
    p.want *= std::max<int64_t>(1, (4 * a.batch + p.want - 1) / p.want);
    if (ragged && a.batch <= 64 && groups * ((p.chunks + 1) / 2) > cus && a.batch * p.chunks < (int64_t)1 << 30) {
        p.segs = p.per = 0;
        p.all = std::min(p.want + a.batch, a.batch * ((p.chunks + 1) / 2));
        return p;
    }
    p.segs = std::max<int64_t>(1, std::min((cus * (ragged ? 4 : 1) + groups - 1) / groups, p.chunks / 2));
    p.per = (p.chunks + p.segs - 1) / p.segs;
    p.segs = (p.chunks + p.per - 1) / p.per;
    p.all = a.batch * p.segs;
    return p;
}

size_t rec_bytes(const Plan& p) { return p.np == 32 ? Rec<32>::bytes : p.np == 64 ? Rec<64>::bytes : Rec<128>::bytes; }
size_t all_rec_bytes(const M2ConvArgs& a, const Plan& p) { return host::align256((size_t)(a.batch * p.chunks * a.G) * rec_bytes(p)); }
size_t seg_bytes(const M2ConvArgs& a, const Plan& p) {
    return p.all == a.batch ? 0 : host::align256((size_t)(p.all * a.H) * (size_t)(a.P * a.N) * 4);
}

struct Run {
    const M2ConvArgs& a;
    const Plan& pl;
    char* recs;
    float *seg_state, *seg_log;
    hipStream_t stream;

    template <typename Tin, typename Tout, int K, int NP, int CT, bool STATE>
    hipError_t pass() const {
        constexpr int bytes = (int)sizeof(Smem<NP, CT>);
        static_assert(bytes <= 160 * 1024, "LDS of a workgroup");
        const auto kern = &m2_chunk_kernel<Tin, Tout, K, NP, CT, STATE>;
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
        const int64_t segs = (pl.all * a.G + 7) / 8 * 8;
        KTime kt(STATE ? "m2_chunk_state" : "m2_chunk_scan", stream);
        hipLaunchKernelGGL(kern, io::groups(segs * pl.sets), dim3(64 * pl.waves), bytes, stream, a, pl, recs, seg_state, seg_log);
        return hipGetLastError();
    }
    template <typename Tin, typename Tout, int K, int NP, int CT>
    hipError_t run() const {
        if (pl.all > a.batch) {
            hipError_t e = pass<Tin, float, K, NP, CT, true>();
            if (e != hipSuccess) return e;
            KTime kt("m2_carry", stream);
            hipLaunchKernelGGL(m2_carry_kernel, io::groups((a.batch * a.H * a.P * a.N / 4 + 255) / 256), dim3(256), 0, stream, a, pl,
                               seg_state, seg_log);
        }
        return pass<Tin, Tout, K, NP, CT, false>();
    }
    template <typename Tin, typename Tout, int K, int NP>
    hipError_t two_blocks() const {
        if constexpr (sizeof(Tin) == 2 || NP < 128) return run<Tin, Tout, K, NP, 2>();
        else return hipErrorInvalidValue;
    }
    template <typename Tin, typename Tout, int K, int NP>
    hipError_t by_ct() const { return pl.ct == 1 ? run<Tin, Tout, K, NP, 1>() : two_blocks<Tin, Tout, K, NP>(); }
    template <typename Tin, typename Tout, int K>
    hipError_t by_np() const {
        return pl.np == 32 ? by_ct<Tin, Tout, K, 32>() : pl.np == 64 ? by_ct<Tin, Tout, K, 64>() : by_ct<Tin, Tout, K, 128>();
    }
    template <typename Tin, typename Tout>
    hipError_t by_k() const {
        return a.conv.K == 2 ? by_np<Tin, Tout, 2>() : a.conv.K == 3 ? by_np<Tin, Tout, 3>() : by_np<Tin, Tout, 4>();
    }
};

}  // namespace

size_t m2_chunk_bytes(const M2ConvArgs& a, int in_bf16) {
    Plan p = plan_of(a, in_bf16, true);
    p.all = std::max(p.all, plan_of(a, in_bf16, false).all);   // (with lengths and without)
    return all_rec_bytes(a, p) + seg_bytes(a, p) + (p.all == a.batch ? 0 : host::align256((size_t)(p.all * a.H) * 4));
}

hipError_t launch_m2_chunk(const M2ConvArgs& a, int in_bf16, int out_bf16, void* ws, hipStream_t stream) {
    const Plan p = plan_of(a, in_bf16, a.conv.lengths != nullptr);
    char* recs = static_cast<char*>(ws);
    char* states = recs + all_rec_bytes(a, p);
    const Run r{a, p, recs, reinterpret_cast<float*>(states), reinterpret_cast<float*>(states + seg_bytes(a, p)), stream};
    const hipError_t e = launch_m2_prep(a, in_bf16, out_bf16, p.np, recs, p.chunks, stream);
    if (e != hipSuccess) return e;
    if (in_bf16) return out_bf16 ? r.by_k<uint16_t, uint16_t>() : r.by_k<uint16_t, float>();
    return out_bf16 ? r.by_k<float, uint16_t>() : r.by_k<float, float>();
}

}  // namespace selscan
