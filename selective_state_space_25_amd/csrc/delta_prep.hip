// delta_prep.hip -- per-chunk matrices of the gated delta rule.
//
// Inside a 64-token chunk, with cum_t the running sum of g and
// G[t, s] = e^(cum_t - cum_s), the errors that the tokens write satisfy a
// unit lower triangular system (see delta_scan.hip), so that the scan needs
//
//   T = (I + M)^-1,  M[t, s] = beta_t G[t, s] k_t.k_s   (s < t)
//   A[t, s] = G[t, s] q_t.k_s                           (s <= t)
//
// which depend on the chunk alone: one workgroup per (batch, head, chunk), all
// in parallel.  The products run on the matrix cores, fp32-grade
// (split_mfma.hpp).  The inverse is blocked: the four 16 x 16 diagonal blocks
// by forward substitution, one per wave; then pairs of blocks, then pairs of
// pairs, joined by -T22 M21 T11 in fp32 MFMAs.  Unlike a series in powers of
// M it stays as exact as substitution when keys repeat.
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

constexpr int kRowM = kC + 4;

template <typename Tin, int NP>
struct PrepSmem {
    static constexpr int kRow = NP + 8;
    uint16_t K[kPlanes<Tin>][kC][kRow];
    uint16_t Q[kPlanes<Tin>][kC][kRow];
    float M[kC][kRowM];
    float T[kC][kRowM];
    double cum[kC];
    float beta[kC];
};

// c + X[r0 + i][c0 + k] Y, Y a 16 x 16 block held as a C tile (rows 4 g + q):
// step q contracts rows 4 g + q, so X is read at columns c0 + 4 g + q.
__device__ __forceinline__ f32x4 mul_block(const float* X, f32x4 y, f32x4 c, int li, int lg) {
    const float4 x = *reinterpret_cast<const float4*>(X + li * kRowM + 4 * lg);
    c = mfma_f32(x.x, y[0], c);
    c = mfma_f32(x.y, y[1], c);
    c = mfma_f32(x.z, y[2], c);
    return mfma_f32(x.w, y[3], c);
}

__device__ __forceinline__ f32x4 ld_block(const float* Y, int li, int lg) {
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = Y[(4 * lg + q) * kRowM + li];
    return v;
}

// GRAD: the transposed blocks too.
template <typename Tin, int NP, bool GRAD>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, float* recs, int64_t nch) {
    constexpr int NK = kPlanes<Tin>;
    constexpr int kRow = PrepSmem<Tin, NP>::kRow;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<PrepSmem<Tin, NP>*>(smem_raw);
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int64_t bh = blockIdx.x / nch, c = blockIdx.x - bh * nch;
    const int64_t b = bh / a.H, h = bh - b * a.H, grp = h / (a.H / a.G);
    const int64_t t0 = c * kC;
    const int64_t len = seq_len(a, b);
    if (t0 >= len) return;
    const int live = (int)min((int64_t)kC, len - t0);
    float* rec = recs + (int64_t)blockIdx.x * (GRAD ? kRecGrad : kRec);

    {   // K and Q rows
        constexpr int ES = (int)sizeof(Tin);
        const int64_t sk = a.G * a.qk_row * ES, at = (b * a.L + t0) * sk + grp * a.qk_row * ES;
        const auto kb = rows_buf(static_cast<const char*>(a.k) + at, live, sk, a.NL * ES);
        const auto qb = rows_buf(static_cast<const char*>(a.q) + at, live, sk, a.NL * ES);
        Raw8<Tin> x[NP / 32], y[NP / 32];
#pragma unroll
        for (int i = 0; i < NP / 32; ++i) {
            const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            const int off = n0 < a.NL ? r * (int)sk + n0 * ES : kOut;
            fetch8(kb, off, x[i]);
            fetch8(qb, off, y[i]);
        }
#pragma unroll
        for (int i = 0; i < NP / 32; ++i) {
            const int id = tid + 256 * i, r = id / (NP / 8), n0 = 8 * (id % (NP / 8));
            stage8(sm.K[0][r], kC * kRow, n0, x[i]);
            stage8(sm.Q[0][r], kC * kRow, n0, y[i]);
        }
    }
    if (wave == 0) {
        const int64_t gi = (b * a.L + t0 + lane) * a.H + h;
        float gv = lane < live ? a.g[gi] : 0.0f;
        const float bv = lane < live ? a.beta[gi] : 0.0f;
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
        rec[kRecGam + lane] = exp_f32((float)cum);
        rec[kRecTail + lane] = exp_f32((float)(last - cum));
        rec[kRecBeta + lane] = bv;
        reinterpret_cast<double*>(rec + kRecCum)[lane] = cum;
    }
    __syncthreads();

    // the 10 lower tiles of K K^T and of Q K^T, five per wave
    for (int id = wave; id < 2 * kBlocks; id += 4) {
        const bool isq = id >= kBlocks;
        const int blk = isq ? id - kBlocks : id;
        int tb, sb;
        lower_tile(blk, tb, sb);
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < NP / 32; ++ks) {
            bf16x8 x[NK], y[NK];
#pragma unroll
            for (int p = 0; p < NK; ++p) {
                x[p] = ld8(isq ? &sm.Q[p][16 * tb + li][32 * ks + 8 * lg] : &sm.K[p][16 * tb + li][32 * ks + 8 * lg]);
                y[p] = ld8(&sm.K[p][16 * sb + li][32 * ks + 8 * lg]);
            }
            acc = mm<3>(x, y, acc);
        }
        const int s = 16 * sb + li;
        const double cs = sm.cum[s];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int t = 16 * tb + 4 * lg + q;
            const float v = acc[q] * exp_f32((float)(sm.cum[t] - cs));
            acc[q] = s <= t ? v : 0.0f;
            if (isq) rec[kRecA + blk * 256 + (4 * lg + q) * 16 + li] = acc[q];
            else sm.M[t][s] = s < t ? sm.beta[t] * v : 0.0f;
        }
        if (GRAD && isq) *reinterpret_cast<f32x4*>(rec + kRecAt + blk * 256 + li * 16 + 4 * lg) = acc;
    }
    __syncthreads();

    {   // diagonal block `wave`: lane's column li by forward substitution
        const int r0 = 16 * wave;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == li ? 1.0f : 0.0f;
            float m[16];
#pragma unroll
            for (int j = 0; j < (i + 3) / 4; ++j) io::ld4(&sm.M[r0 + i][r0 + 4 * j], m + 4 * j);
#pragma unroll
            for (int j = 0; j < i; ++j) v = __builtin_fmaf(-m[j], x[j], v);
            x[i] = v;
        }
        if (lg == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sm.T[r0 + i][r0 + li] = x[i];
        }
    }
    __syncthreads();
    const f32x4 z4 = {0.0f, 0.0f, 0.0f, 0.0f};
    if (wave < 2) {   // blocks (1, 0) and (3, 2)
        const int r0 = 32 * wave + 16, c0 = 32 * wave;
        const f32x4 x = mul_block(&sm.M[r0][c0], ld_block(&sm.T[c0][c0], li, lg), z4, li, lg);
        const f32x4 t = mul_block(&sm.T[r0][r0], x, z4, li, lg);
#pragma unroll
        for (int q = 0; q < 4; ++q) sm.T[r0 + 4 * lg + q][c0 + li] = -t[q];
    }
    __syncthreads();
    {   // block (2 + rb, cb) of -T[2.., 2..] (M[2.., 0..] T[0.., 0..])
        const int rb = wave >> 1, cb = wave & 1;
        f32x4 t = z4;
        for (int i = 0; i <= rb; ++i) {
            f32x4 x = z4;
            for (int j = cb; j < 2; ++j)
                x = mul_block(&sm.M[32 + 16 * i][16 * j], ld_block(&sm.T[16 * j][16 * cb], li, lg), x, li, lg);
            t = mul_block(&sm.T[32 + 16 * rb][32 + 16 * i], x, t, li, lg);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) sm.T[32 + 16 * rb + 4 * lg + q][16 * cb + li] = -t[q];
    }
    __syncthreads();
    for (int i = tid; i < kBlocks * 64; i += 256) {
        int tb, sb;
        lower_tile(i >> 6, tb, sb);
        const int r = (i & 63) >> 2, q4 = 4 * (i & 3);
        *reinterpret_cast<float4*>(rec + kRecT + 4 * i) =
            *reinterpret_cast<const float4*>(&sm.T[16 * tb + r][16 * sb + q4]);
        if constexpr (GRAD) {
            const float* x = &sm.T[16 * tb + q4][16 * sb + r];
            *reinterpret_cast<float4*>(rec + kRecTt + 4 * i) = make_float4(x[0], x[kRowM], x[2 * kRowM], x[3 * kRowM]);
        }
    }
}

template <typename Tin, int NP, bool GRAD>
hipError_t launch(const DeltaArgs& a, float* recs, int64_t nch, hipStream_t stream) {
    const auto kern = &delta_prep_kernel<Tin, NP, GRAD>;
    constexpr int bytes = (int)sizeof(PrepSmem<Tin, NP>);
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    KTime kt("delta_prep", stream);
    hipLaunchKernelGGL(kern, dim3((unsigned)(a.batch * a.H * nch)), dim3(256), bytes, stream, a, recs, nch);
    return hipGetLastError();
}

template <typename Tin, bool GRAD>
hipError_t by_n(const DeltaArgs& a, float* recs, hipStream_t stream) {
    const int64_t nch = delta_chunks(a.L);
    return a.N <= 64 ? launch<Tin, 64, GRAD>(a, recs, nch, stream) : launch<Tin, 128, GRAD>(a, recs, nch, stream);
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
size_t delta_record_bytes(bool grad) { return sizeof(float) * (grad ? dchunk::kRecGrad : dchunk::kRec); }

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

hipError_t launch_delta_prep(const DeltaArgs& a, int in_bf16, bool grad, float* recs, hipStream_t stream) {
    if (in_bf16) return grad ? by_n<uint16_t, true>(a, recs, stream) : by_n<uint16_t, false>(a, recs, stream);
    return grad ? by_n<float, true>(a, recs, stream) : by_n<float, false>(a, recs, stream);
}

}  // namespace selscan
