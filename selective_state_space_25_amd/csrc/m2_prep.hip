// m2_prep.hip -- B and C of the Mamba-2 mixer's chunks, for gfx950.
//
// Per (batch, 64-token chunk, group): the short convolution with silu of the
// group's 2 N channels of B and C in fp32, split into three bf16 planes
// (split_mfma.hpp) and laid out as the scan's operands (m2_chunk.hpp), and
// G = C B^T on and below the diagonal, which the heads of the group share.  A
// thread has two neighbouring channels and walks 16 tokens (N = 128; fewer
// for smaller N) with the last K - 1 inputs in registers; eight consecutive
// tokens of a channel are an operand of B^T as they are, the others are turned
// in LDS.
//
// 1 x 16384, one group, N = 128: 21 us, 28 MB of records written.  A workgroup
// a chunk is 256 of them, one a compute unit: its chain of loads, convolution,
// splits and products is what takes the time (waves wait 57 % of it).
#include "m2_chunk.hpp"

namespace selscan {

namespace {

using namespace m2chunk;

constexpr int kT = 512;

template <int NP>
struct Smem {
    static constexpr int kRow = NP + 8;
    uint16_t p[2][3][kC][kRow];   // B, C; planes; tokens; n in operand order
    __attribute__((aligned(16))) float g[8][16 * 36];
};

// Where n stands in its row: the operands' order within each 32.
__device__ __forceinline__ int place(int n) { return (n & ~31) + 8 * ((n & 15) >> 2) + 4 * ((n & 31) >> 4) + (n & 3); }

template <typename Tin, int K, int NP>
__global__ __launch_bounds__(kT) void m2_prep_kernel(M2ConvArgs a, int y_bytes, char* recs, int64_t chunks) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<Smem<NP>*>(smem_raw);
    constexpr int kSlices = NP == 32 ? 8 : kT / NP, kTokens = kC / kSlices;   // of a thread's two channels
    const int tid = threadIdx.x;
    const int64_t id = io::group_id();
    const int64_t bc = id / a.G, g = id - bc * a.G, b = bc / chunks, c = bc - b * chunks;
    if (b >= a.batch) return;
    const int64_t len = seq_len(a, b), t0 = c * kC;
    const int64_t C = a.conv.C, row = a.conv.x_row;
    const Tin* X = static_cast<const Tin*>(a.conv.x) + b * a.conv.x_batch;
    const Tin* S = a.conv.state ? static_cast<const Tin*>(a.conv.state) + b * (K - 1) * C : nullptr;
    if (c == 0 && g == 0 && a.conv.last) {
        // the convolution's state after the sequence, all channels
        for (int64_t e = tid; e < C * (K - 1); e += kT) {
            const int64_t j = e / C, ch = e - j * C, t = len - (K - 1) + j;
            Tin v = Tin(0);
            if (t >= 0) v = X[t * row + ch];
            else if (S) v = S[(t + K - 1) * C + ch];
            static_cast<Tin*>(a.conv.last)[b * (K - 1) * C + e] = v;
        }
    }
    if (t0 >= len) {
        // past the end: the group's y are zero
        const int64_t n = a.H / a.G * a.P * y_bytes / 2, pieces = (n + 7) / 8, rows = min((int64_t)kC, a.L - t0);
        uint16_t* Y = static_cast<uint16_t*>(a.y) + ((b * a.L + t0) * a.G + g) * n;
        io::Piece<uint16_t, 8> none;
        none.zero();
        for (int64_t e = tid; e < rows * pieces; e += kT) {
            const int64_t t = e / pieces, d = 8 * (e - t * pieces);
            uint16_t* to = Y + t * a.G * n + d;
            if (d + 8 <= n) none.put(to);
            else
                for (int i = 0; i < n - d; ++i) to[i] = 0;
        }
        return;
    }
    char* rec = recs + id * Rec<NP>::bytes;
    {
        const int ch = 2 * (tid % NP), isC = ch >= NP, n = ch % NP, first = tid / NP * kTokens;
        const bool live = n < a.N && first < kC;
        const int64_t cc = a.H * a.P + (isC * a.G + g) * a.N + (live ? n : 0);
        float w[K][2], bias[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bias[i] = a.conv.bias ? a.conv.bias[cc + i] : 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][i] = a.conv.weight[(cc + i) * K + k];
        }
        auto input = [&](int64_t t, float (&v)[2]) {
            io::Piece<Tin, 2> r;
            r.zero();
            if (live && t < len) {
                if (t >= 0) r.get(X + t * row + cc);
                else if (S) r.get(S + (t + K - 1) * C + cc);
            }
            r.widen(v);
        };
        float xs[K - 1 + kTokens][2];
#pragma unroll
        for (int j = 0; j < K - 1 + kTokens; ++j) input(t0 + first - (K - 1) + j, xs[j]);
        uint16_t* to = &sm.p[isC][0][0][place(n)];
#pragma unroll
        for (int t = 0; t < kTokens; t += 8) {
            if (first >= kC) break;
            u32x4 p[3][2];   // planes of the eight tokens' channel pairs
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v[2];
                const bool in = live && t0 + first + t + j < len;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float pre = bias[i];
#pragma unroll
                    for (int k = 0; k < K; ++k) pre = __builtin_fmaf(w[k][i], xs[t + j + k][i], pre);
                    v[i] = in ? silu_scaled(pre, 1.0f) : 0.0f;
                }
                u32x4 q[3];
                split2<3>(v[0], v[1], q, 0);
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    p[x][j >> 2][j & 3] = q[x][0];
                    *reinterpret_cast<uint32_t*>(to + (x * kC + first + t + j) * Smem<NP>::kRow) = q[x][0];
                }
            }
            if (isC) continue;
            const int tok = first + t;
#pragma unroll
            for (int x = 0; x < 3; ++x)
#pragma unroll
                for (int i = 0; i < 2; ++i) {   // the eight tokens of one channel
                    u32x4 o;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = __builtin_amdgcn_perm(p[x][e >> 1][2 * (e & 1) + 1], p[x][e >> 1][2 * (e & 1)], i ? 0x07060302 : 0x05040100);
                    *reinterpret_cast<u32x4*>(rec + Rec<NP>::B + (((n >> 4) * 2 + (tok >> 5)) * 3 + x) * kBlock +
                                              (((tok >> 3) & 3) * 16 + (n & 15) + i) * 16) = o;
                }
        }
    }
    __syncthreads();
    // G: a wave has the columns 32 ks .. of rows 16 tt ..
    const int lane = tid & 63, li = lane & 15, lg = lane >> 4, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tt = wave >> 1, half = wave & 1;
    f32x4 acc[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) acc[s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < NP / 32; ++ks) {
        bf16x8 cp[3], bp[2][3];
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            cp[x] = ld8(&sm.p[1][x][16 * tt + li][32 * ks + 8 * lg]);
            if (half == (ks & 1)) *reinterpret_cast<bf16x8*>(rec + ((ks * 4 + tt) * 3 + x) * kBlock + lane * 16) = cp[x];
        }
        if (2 * half > tt) continue;   // (the store above is the other half's too)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int x = 0; x < 3; ++x) bp[s][x] = ld8(&sm.p[0][x][32 * half + 16 * s + li][32 * ks + 8 * lg]);
        mm_turns<3, 3, 3>([&](int) -> const bf16x8(&)[3] { return cp; }, [&](int m) -> const bf16x8(&)[3] { return bp[m]; }, acc);
    }
    if (2 * half > tt) return;
    // through LDS into operand order, zero above the diagonal
    float* to = sm.g[wave];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int t = 4 * lg + q, col = 16 * s + li;   // row 16 tt + t, column 32 half + col
            to[t * 36 + col] = 32 * half + col <= 16 * tt + t ? acc[s][q] : 0.0f;
        }
    dchunk::wave_sync();
    const float* from = to + li * 36 + 8 * lg;
    bf16x8 gp[3];
    split8<3>(*reinterpret_cast<const f32x4*>(from), *reinterpret_cast<const f32x4*>(from + 4), gp);
#pragma unroll
    for (int x = 0; x < 3; ++x)
        *reinterpret_cast<bf16x8*>(rec + Rec<NP>::G + (g_tile(tt, half) * 3 + x) * kBlock + lane * 16) = gp[x];
}

template <typename Tin, int K, int NP>
hipError_t launch(const M2ConvArgs& a, int y_bytes, char* recs, int64_t chunks, hipStream_t stream) {
    constexpr int bytes = (int)sizeof(Smem<NP>);
    const auto kern = &m2_prep_kernel<Tin, K, NP>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    KTime kt("m2_prep", stream);
    hipLaunchKernelGGL(kern, io::groups(a.batch * chunks * a.G), dim3(kT), bytes, stream, a, y_bytes, recs, chunks);
    return hipGetLastError();
}

template <typename Tin, int K>
hipError_t by_np(const M2ConvArgs& a, int y_bytes, int np, char* recs, int64_t chunks, hipStream_t st) {
    return np == 32 ? launch<Tin, K, 32>(a, y_bytes, recs, chunks, st) : np == 64 ? launch<Tin, K, 64>(a, y_bytes, recs, chunks, st)
                                                                        : launch<Tin, K, 128>(a, y_bytes, recs, chunks, st);
}

template <typename Tin>
hipError_t by_k(const M2ConvArgs& a, int y_bytes, int np, char* recs, int64_t chunks, hipStream_t st) {
    return a.conv.K == 2 ? by_np<Tin, 2>(a, y_bytes, np, recs, chunks, st) : a.conv.K == 3 ? by_np<Tin, 3>(a, y_bytes, np, recs, chunks, st)
                                                                                 : by_np<Tin, 4>(a, y_bytes, np, recs, chunks, st);
}

}  // namespace

hipError_t launch_m2_prep(const M2ConvArgs& a, int in_bf16, int out_bf16, int np, char* recs, int64_t chunks, hipStream_t stream) {
    const int y_bytes = out_bf16 ? 2 : 4;
    return in_bf16 ? by_k<uint16_t>(a, y_bytes, np, recs, chunks, stream) : by_k<float>(a, y_bytes, np, recs, chunks, stream);
}

}  // namespace selscan
