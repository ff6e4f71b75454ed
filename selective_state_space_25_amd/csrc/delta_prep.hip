// delta_prep.hip -- per-chunk matrices of the gated delta rule.
//
// Inside a 64-token chunk, with cum_t the running sum of g and
// G[t, s] = e^(cum_t - cum_s), the errors that the tokens write satisfy a
// unit lower triangular system (see delta_scan.hip), so that the scan needs
//
//   T = (I + M)^-1,  M[t, s] = beta_t G[t, s] k_t.k_s   (s < t)
//   A[t, s] = G[t, s] q_t.k_s                           (s <= t)
//
// which depend on the chunk alone.  One wave per (batch, head, chunk), with
// no barrier anywhere: K K^T and Q K^T on the matrix cores, fp32-grade
// (split_mfma.hpp), the wave's lanes reading K and Q rows straight into
// operands (a row block is the same registers as A and as B operand); then
// the inverse in LDS, in place, blocked: the four 16 x 16 diagonal blocks by
// forward substitution, a lane group each; then pairs of blocks, then pairs
// of pairs, joined by -T22 M21 T11 in fp32 MFMAs.  Unlike a series in powers
// of M it stays as exact as substitution when keys repeat.  T and A leave
// already split into the planes that the scan multiplies with.
//
// What bounds it are the records (32 KB a chunk and head, 57.6 KB for the
// gradients) and the inverse's chain of dependent steps:
// 16 heads of 128, L 16384: 64 us, 131 MB of records and 134 MB of q and k,
// 4.1 TB/s; 256 heads, L 4096, q and k shared by 32 of them: 149 us, 524 MB of
// records, 3.5 TB/s.
//
// cum is summed in fp64 and G's exponents are fp64 differences: after a
// strong decay cum is large and its fp32 steps would be errors of the
// decays between the tokens that follow.  g below -200 counts as -200, whose
// exponential is zero in fp32 either way, so that a reset (-inf) stays finite.
#include <algorithm>

#include "delta_chunk.hpp"

namespace selscan {

namespace {

using namespace dchunk;

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

constexpr int kRowB = 20;    // padded row of a 16 x 16 block
constexpr int kUnits = 4;    // waves per workgroup

struct PrepUnit {
    float M[kBlocks][16][kRowB];   // A's blocks, then M's, then T's
    double cum[kC];
    float beta[kC];
};

// c + X Y: X a block in LDS, Y a block held as a C tile (rows 4 g + q); step
// q contracts rows 4 g + q, so X is read at columns 4 g + q.
__device__ __forceinline__ f32x4 mul_block(const float (&X)[16][kRowB], f32x4 y, f32x4 c, int li, int lg) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(&X[li][4 * lg]);
#pragma unroll
    for (int q = 0; q < 4; ++q) c = mfma_f32(x[q], y[q], c);
    return c;
}

__device__ __forceinline__ f32x4 ld_block(const float (&Y)[16][kRowB], int li, int lg) {
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = Y[4 * lg + q][li];
    return v;
}

__device__ __forceinline__ void st_block(float (&Y)[16][kRowB], f32x4 v, int li, int lg) {
#pragma unroll
    for (int q = 0; q < 4; ++q) Y[4 * lg + q][li] = v[q];
}

// GRAD: the gradients' record.
template <typename Tin, int NP, bool GRAD>
__global__ __launch_bounds__(64 * kUnits) void delta_prep_kernel(DeltaArgs a, char* recs, int64_t nch, int64_t units) {
    constexpr int NK = kPlanes<Tin>, ES = (int)sizeof(Tin);
    using R = Rec<GRAD>;
    __shared__ __attribute__((aligned(16))) PrepUnit sms[kUnits];
    PrepUnit& sm = sms[threadIdx.x >> 6];
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
    const int64_t unit = (int64_t)blockIdx.x * kUnits + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (unit >= units) return;
    const int64_t bh = unit / nch, c = unit - bh * nch;
    const int64_t b = bh / a.H, h = bh - b * a.H, grp = h / (a.H / a.G);
    const int64_t t0 = c * kC;
    const int64_t len = seq_len(a, b);
    if (t0 >= len) return;
    const int live = (int)min((int64_t)kC, len - t0);
    char* rec = recs + unit * R::bytes;

    const int64_t gi = (b * a.L + t0 + lane) * a.H + h;
    float gv = lane < live ? a.g[gi] : 0.0f;
    const float bv = lane < live ? a.beta[gi] : 0.0f;

    // the 10 lower tiles of K K^T and of Q K^T
    f32x4 kk[kBlocks], qk[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) kk[i] = qk[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    {
        const int sk = scalar((int)(a.G * a.qk_row * ES));
        const int64_t at = (b * a.L + t0) * sk + grp * a.qk_row * ES;
        const auto kb = rows_buf(scalar(static_cast<const char*>(a.k) + at), scalar(live), sk, a.NL * ES);
        const auto qb = rows_buf(scalar(static_cast<const char*>(a.q) + at), scalar(live), sk, a.NL * ES);
#pragma unroll
        for (int ks = 0; ks < NP / 32; ++ks) {
            const int n = 32 * ks + 8 * lg;
            bf16x8 k[4][NK], q[4][NK];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int off = n < a.NL ? (16 * t + li) * sk + n * ES : kOut;
                Raw8<Tin> x, y;
                fetch8(kb, off, x);
                fetch8(qb, off, y);
                to_operand(x, k[t]);
                to_operand(y, q[t]);
            }
#pragma unroll
            for (int s = 2; s >= 0; --s)
#pragma unroll
                for (int i = 0; i < NK; ++i)
                    if (s - i >= 0 && s - i < NK) {
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int u = 0; u <= t; ++u) {
                                kk[block_at(t, u)] = mfma(k[t][i], k[u][s - i], kk[block_at(t, u)]);
                                qk[block_at(t, u)] = mfma(q[t][i], k[u][s - i], qk[block_at(t, u)]);
                            }
                    }
        }
    }
    gv = gv < -200.0f ? -200.0f : gv;   // (a NaN stays)
    double cum = gv;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double up = __shfl_up(cum, o, 64);
        if (lane >= o) cum += up;
    }
    const double last = __shfl(cum, 63, 64);
    sm.cum[lane] = cum;
    sm.beta[lane] = bv;
    reinterpret_cast<float*>(rec + R::gam)[lane] = exp_f32((float)cum);
    reinterpret_cast<float*>(rec + R::tail)[lane] = exp_f32((float)(last - cum));
    reinterpret_cast<float*>(rec + R::beta)[lane] = bv;
    reinterpret_cast<double*>(rec + R::cum)[lane] = cum;

    wave_sync();
    // A; M in kk
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        double ct[4];
        f32x4 bt = *reinterpret_cast<const f32x4*>(&sm.beta[16 * t + 4 * lg]);
#pragma unroll
        for (int q = 0; q < 4; ++q) ct[q] = sm.cum[16 * t + 4 * lg + q];
#pragma unroll
        for (int s = 0; s <= t; ++s) {
            const int i = block_at(t, s);
            const double cs = sm.cum[16 * s + li];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float g = exp_f32((float)(ct[q] - cs));
                if (s == t && li > 4 * lg + q) g = 0.0f;
                // (a select, not a product with zero: what is above the diagonal may not be finite)
                qk[i][q] = s == t && li > 4 * lg + q ? 0.0f : g * qk[i][q];
                kk[i][q] = s == t && li >= 4 * lg + q ? 0.0f : bt[q] * g * kk[i][q];
            }
            if constexpr (GRAD) {
                uint2 w[3];
                split4<3>(qk[i], w);
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    *reinterpret_cast<uint2*>(rec + R::At + x * kPlane + i * 512 + li * 32 + lg * 8) = w[x];
                float* f = reinterpret_cast<float*>(rec + R::A) + i * 256 + 64 * lg + li;
#pragma unroll
                for (int q = 0; q < 4; ++q) f[16 * q] = qk[i][q];
            } else {
                st_block(sm.M[i], qk[i], li, lg);
            }
        }
    }
    // the blocks in LDS to planes, a lane eight columns of a row of a pair of blocks
    const int r8 = (lane & 31) >> 1, c8 = 8 * (lane & 1);
    auto put_planes = [&](char* to) {
#pragma unroll
        for (int i = 0; i < kBlocks; i += 2) {
            const float* x = &sm.M[i + (lane >> 5)][r8][c8];
            bf16x8 w[3];
            split8<3>(*reinterpret_cast<const f32x4*>(x), *reinterpret_cast<const f32x4*>(x + 4), w);
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(to + p * kPlane + i * 512 + lane * 16) = w[p];
        }
    };
    wave_sync();
    if constexpr (!GRAD) put_planes(rec + R::A);
    wave_sync();
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) st_block(sm.M[i], kk[i], li, lg);
    wave_sync();

    {   // diagonal block lg, column li
        float (&D)[16][kRowB] = sm.M[block_at(lg, lg)];
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == li ? 1.0f : 0.0f;
            float m[16];
#pragma unroll
            for (int j = 0; j < (i + 3) / 4; ++j) io::ld4(&D[i][4 * j], m + 4 * j);
#pragma unroll
            for (int j = 0; j < i; ++j) v = __builtin_fmaf(-m[j], x[j], v);
            x[i] = v;
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < 16; ++i) D[i][li] = x[i];
    }
    wave_sync();
    const f32x4 z4 = {0.0f, 0.0f, 0.0f, 0.0f};
    auto M = [&](int t, int s) -> float (&)[16][kRowB] { return sm.M[block_at(t, s)]; };
    {   // blocks (1, 0) and (3, 2)
        const f32x4 x0 = mul_block(M(1, 0), ld_block(M(0, 0), li, lg), z4, li, lg);
        const f32x4 x1 = mul_block(M(3, 2), ld_block(M(2, 2), li, lg), z4, li, lg);
        const f32x4 t0_ = mul_block(M(1, 1), x0, z4, li, lg);
        const f32x4 t1_ = mul_block(M(3, 3), x1, z4, li, lg);
        wave_sync();
        st_block(M(1, 0), -t0_, li, lg);
        st_block(M(3, 2), -t1_, li, lg);
    }
    wave_sync();
    {   // blocks (2 .. 3, 0 .. 1)
        const f32x4 y00 = ld_block(M(0, 0), li, lg), y10 = ld_block(M(1, 0), li, lg), y11 = ld_block(M(1, 1), li, lg);
        f32x4 x00 = mul_block(M(2, 0), y00, z4, li, lg), x10 = mul_block(M(3, 0), y00, z4, li, lg);
        const f32x4 x01 = mul_block(M(2, 1), y11, z4, li, lg), x11 = mul_block(M(3, 1), y11, z4, li, lg);
        x00 = mul_block(M(2, 1), y10, x00, li, lg);
        x10 = mul_block(M(3, 1), y10, x10, li, lg);
        const f32x4 t20 = mul_block(M(2, 2), x00, z4, li, lg), t21 = mul_block(M(2, 2), x01, z4, li, lg);
        f32x4 t30 = mul_block(M(3, 2), x00, z4, li, lg), t31 = mul_block(M(3, 2), x01, z4, li, lg);
        t30 = mul_block(M(3, 3), x10, t30, li, lg);
        t31 = mul_block(M(3, 3), x11, t31, li, lg);
        wave_sync();
        st_block(M(2, 0), -t20, li, lg);
        st_block(M(2, 1), -t21, li, lg);
        st_block(M(3, 0), -t30, li, lg);
        st_block(M(3, 1), -t31, li, lg);
    }
    wave_sync();
    put_planes(rec + R::T);
    if constexpr (GRAD) {
#pragma unroll
        for (int i = 0; i < kBlocks; i += 2) {   // row r8 of the transposed block: column r8 down
            const float* x = &sm.M[i + (lane >> 5)][c8][r8];
            f32x4 lo, hi;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                lo[q] = x[q * kRowB];
                hi[q] = x[(4 + q) * kRowB];
            }
            bf16x8 w[3];
            split8<3>(lo, hi, w);
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(rec + R::Tt + p * kPlane + i * 512 + lane * 16) = w[p];
        }
    }
}

template <typename Tin, int NP, bool GRAD>
hipError_t launch(const DeltaArgs& a, char* recs, hipStream_t stream) {
    const int64_t nch = delta_chunks(a.L), units = a.batch * a.H * nch;
    KTime kt("delta_prep", stream);
    hipLaunchKernelGGL((delta_prep_kernel<Tin, NP, GRAD>), dim3((unsigned)((units + kUnits - 1) / kUnits)),
                       dim3(64 * kUnits), 0, stream, a, recs, nch, units);
    return hipGetLastError();
}

template <typename Tin, bool GRAD>
hipError_t by_n(const DeltaArgs& a, char* recs, hipStream_t stream) {
    return a.N <= 64 ? launch<Tin, 64, GRAD>(a, recs, stream) : launch<Tin, 128, GRAD>(a, recs, stream);
}

template <typename Tin>
hipError_t by_use(const DeltaArgs& a, bool grad, char* recs, hipStream_t stream) {
    return grad ? by_n<Tin, true>(a, recs, stream) : by_n<Tin, false>(a, recs, stream);
}

// Rows of N elements, one after the other, to rows of `to`, zeros past N.
template <typename T>
__global__ __launch_bounds__(256) void delta_pad_kernel(const T* q, const T* k, T* qo, T* ko, int N, int to, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / to;
        const int c = (int)(i - r * to);
        qo[i] = c < N ? q[r * N + c] : T(0);
        ko[i] = c < N ? k[r * N + c] : T(0);
    }
}

}  // namespace

int64_t delta_chunks(int64_t L) { return (L + dchunk::kC - 1) / dchunk::kC; }
size_t delta_record_bytes(bool grad) { return grad ? dchunk::GradRec::bytes : dchunk::Rec<false>::bytes; }

hipError_t launch_delta_pad(DeltaArgs& a, int in_bf16, void* rows, hipStream_t stream) {
    const int to = a.N <= 64 ? 64 : 128;
    const int64_t n = a.batch * a.L * a.G * to;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 1 << 16);
    KTime kt("delta_pad", stream);
    void* k = static_cast<char*>(rows) + n * (in_bf16 ? 2 : 4);
    if (in_bf16)
        hipLaunchKernelGGL((delta_pad_kernel<uint16_t>), dim3(blocks), dim3(256), 0, stream,
                           static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.k),
                           static_cast<uint16_t*>(rows), static_cast<uint16_t*>(k), a.N, to, n);
    else
        hipLaunchKernelGGL((delta_pad_kernel<float>), dim3(blocks), dim3(256), 0, stream, static_cast<const float*>(a.q),
                           static_cast<const float*>(a.k), static_cast<float*>(rows), static_cast<float*>(k), a.N, to, n);
    a.q = rows;
    a.k = k;
    a.NL = to;
    a.qk_row = to;
    return hipGetLastError();
}

hipError_t launch_delta_prep(const DeltaArgs& a, int in_bf16, bool grad, char* recs, hipStream_t stream) {
    return in_bf16 ? by_use<uint16_t>(a, grad, recs, stream) : by_use<float>(a, grad, recs, stream);
}

}  // namespace selscan
