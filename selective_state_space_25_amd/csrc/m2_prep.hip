// m2_prep.hip -- B and C of the Mamba-2 mixer's chunks, for gfx950.
//
// Per (batch, 64-token chunk, group): the short convolution with silu of the
// group's 2 N channels of B and C in fp32, split into three bf16 planes
// (split_mfma.hpp) and laid out as the scan's operands (m2_chunk.hpp), and
// G = C B^T, which the heads of the group share.  A thread has one channel and
// walks its tokens with the last K - 1 inputs in registers; eight consecutive
// tokens of it are an operand of B^T as they are, the others are turned in LDS.
#include "m2_chunk.hpp"

namespace selscan {

namespace {

using namespace m2chunk;

constexpr int kT = 256;

template <int NP>
struct Smem {
    static constexpr int kRow = NP + 8;
    uint16_t p[2][3][kC][kRow];   // B, C; planes; tokens; n in operand order
};

// Where n stands in its row: the operands' order within each 32.
__device__ __forceinline__ int place(int n) { return (n & ~31) + 8 * ((n & 15) >> 2) + 4 * ((n & 31) >> 4) + (n & 3); }

template <typename Tin, int K, int NP>
__global__ __launch_bounds__(kT) void m2_prep_kernel(M2ConvArgs a, char* recs, int64_t chunks) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<Smem<NP>*>(smem_raw);
    constexpr int kSlices = kT / (2 * NP), kTokens = kC / kSlices;   // of a thread
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
    if (t0 >= len) return;
    char* rec = recs + id * Rec<NP>::bytes;
    {
        const int ch = tid % (2 * NP), isC = ch >= NP, n = ch % NP, first = tid / (2 * NP) * kTokens;
        const bool live = n < a.N;
        const int64_t cc = a.H * a.P + (isC * a.G + g) * a.N + (live ? n : 0);
        float w[K], bias = a.conv.bias ? a.conv.bias[cc] : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = a.conv.weight[cc * K + k];
        auto input = [&](int64_t t) {
            if (!live || t >= len) return 0.0f;
            if (t >= 0) return io::ld(X + t * row + cc);
            return S ? io::ld(S + (t + K - 1) * C + cc) : 0.0f;
        };
        float xs[K - 1 + 8];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) xs[j] = input(t0 + first - (K - 1) + j);
        uint16_t* to = &sm.p[isC][0][0][place(n)];
#pragma unroll 2
        for (int t = first; t < first + kTokens; t += 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) xs[K - 1 + j] = input(t0 + t + j);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float pre = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) pre = __builtin_fmaf(w[k], xs[j + k], pre);
                v[j] = live && t0 + t + j < len ? silu_scaled(pre, 1.0f) : 0.0f;
            }
            u32x4 p[3];
#pragma unroll
            for (int e = 0; e < 4; ++e) split2<3>(v[2 * e], v[2 * e + 1], p, e);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (!isC)
                    *reinterpret_cast<u32x4*>(rec + Rec<NP>::B + (((n >> 4) * 2 + (t >> 5)) * 3 + x) * kBlock +
                                              (((t >> 3) & 3) * 16 + (n & 15)) * 16) = p[x];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    to[(x * kC + t + 2 * e) * Smem<NP>::kRow] = (uint16_t)p[x][e];
                    to[(x * kC + t + 2 * e + 1) * Smem<NP>::kRow] = (uint16_t)(p[x][e] >> 16);
                }
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) xs[j] = xs[8 + j];
        }
    }
    __syncthreads();
    const int lane = tid & 63, li = lane & 15, lg = lane >> 4, tt = __builtin_amdgcn_readfirstlane(tid >> 6);
    f32x4 acc[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < NP / 32; ++ks) {
        bf16x8 cp[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            cp[x] = ld8(&sm.p[1][x][16 * tt + li][32 * ks + 8 * lg]);
            *reinterpret_cast<bf16x8*>(rec + ((ks * 4 + tt) * 3 + x) * kBlock + lane * 16) = cp[x];
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (s <= tt) {
                bf16x8 bp[3];
#pragma unroll
                for (int x = 0; x < 3; ++x) bp[x] = ld8(&sm.p[0][x][16 * s + li][32 * ks + 8 * lg]);
                acc[s] = mm<3>(cp, bp, acc[s]);
            }
    }
    float* G = reinterpret_cast<float*>(rec + Rec<NP>::G);
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (s <= tt) {
#pragma unroll
            for (int q = 0; q < 4; ++q)   // row 16 tt + 4 lg + q, column 16 s + li
                G[g_tile(tt, s >> 1) * 512 + (4 * lg + q + 16 * (2 * (s & 1) + (li >> 3))) * 8 + (li & 7)] = acc[s][q];
        }
}

template <typename Tin, int K, int NP>
hipError_t launch(const M2ConvArgs& a, char* recs, int64_t chunks, hipStream_t stream) {
    constexpr int bytes = (int)sizeof(Smem<NP>);
    const auto kern = &m2_prep_kernel<Tin, K, NP>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    KTime kt("m2_prep", stream);
    hipLaunchKernelGGL(kern, io::groups(a.batch * chunks * a.G), dim3(kT), bytes, stream, a, recs, chunks);
    return hipGetLastError();
}

template <typename Tin, int K>
hipError_t by_np(const M2ConvArgs& a, int np, char* recs, int64_t chunks, hipStream_t st) {
    return np == 32 ? launch<Tin, K, 32>(a, recs, chunks, st) : np == 64 ? launch<Tin, K, 64>(a, recs, chunks, st)
                                                                        : launch<Tin, K, 128>(a, recs, chunks, st);
}

template <typename Tin>
hipError_t by_k(const M2ConvArgs& a, int np, char* recs, int64_t chunks, hipStream_t st) {
    return a.conv.K == 2 ? by_np<Tin, 2>(a, np, recs, chunks, st) : a.conv.K == 3 ? by_np<Tin, 3>(a, np, recs, chunks, st)
                                                                                 : by_np<Tin, 4>(a, np, recs, chunks, st);
}

}  // namespace

hipError_t launch_m2_prep(const M2ConvArgs& a, int in_bf16, int np, char* recs, int64_t chunks, hipStream_t stream) {
    return in_bf16 ? by_k<uint16_t>(a, np, recs, chunks, stream) : by_k<float>(a, np, recs, chunks, stream);
}

}  // namespace selscan
