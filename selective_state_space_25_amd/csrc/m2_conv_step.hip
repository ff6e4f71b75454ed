// m2_conv_step.hip -- one token through the short convolution and the Mamba-2
// state update, for gfx950.
//
//   v = silu(bias + sum_k w[k] xbc_{t-K+1+k});   x, B, C = the parts of v
//   D_t = softplus(dt + dt_bias);   S = exp(D_t A) S + D_t x B^T;   y = S C + D x
//
// The state is read and written once, which bounds a full batch; one sequence
// is the launch.  A workgroup has kRows rows of one head's state for each of R
// turns: it asks for the state first, makes its B, C (2 N channels, the same
// in every workgroup of a group) and x into LDS while those loads are on their
// way, and then updates: the lanes of a row hold 8 (N >= 64) or 4 states each
// and add y up by shuffles.  The convolution's result is never rounded to 16
// bits.  The convolution's state is only read here: the workgroups of a group
// share the channels of B and C, so a kernel behind this one moves it on.
//
// 32 heads of 64 x 128, bf16: batch 128 56 us for 0.27 GB of state read and
// written, 4.8 TB/s, with the launch behind it 59.5; one sequence 4.4 and 2.1
// us, below what the two launches take the host (7.5).
#include "io.hpp"
#include "kernels.hpp"

namespace selscan {

namespace {

constexpr int kT = 256;

template <typename Tin, typename Tout, int K, int N, int R>
__global__ __launch_bounds__(kT) void m2_conv_step_kernel(M2ConvArgs a) {
    constexpr int E = N >= 64 ? 8 : 4;      // states a lane
    constexpr int Q = N / E;                // lanes a row
    constexpr int kRows = kT / Q;
    __shared__ __attribute__((aligned(16))) float Bs[N], Cs[N];
    __shared__ float xs[R * kRows];
    const int64_t pblocks = (a.P + R * kRows - 1) / (R * kRows);
    const int64_t id = io::group_id(), bh = id / pblocks;
    if (bh >= a.batch * a.H) return;
    const int64_t p0 = (id - bh * pblocks) * (R * kRows);
    const int64_t b = bh / a.H, h = bh - b * a.H, g = h / (a.H / a.G);
    const int tid = threadIdx.x, row = tid / Q, q = tid % Q;
    float* S = a.last + (bh * a.P + p0) * N + q * E;
    float s[R][E];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (p0 + r * kRows + row < a.P) {
#pragma unroll
            for (int e = 0; e < E; e += 4) io::ld4(S + (int64_t)(r * kRows + row) * N + e, s[r] + e);
        }
    const int nx = (int)min((int64_t)(R * kRows), a.P - p0);
    for (int i = tid; i < 2 * N + nx; i += kT) {
        const int64_t c = i < 2 * N ? a.H * a.P + (i / N * a.G + g) * N + i % N : h * a.P + p0 + (i - 2 * N);
        const Tin* W = static_cast<const Tin*>(a.conv.state) + b * (K - 1) * a.conv.C + c;
        float v = a.conv.bias ? a.conv.bias[c] : 0.0f;
#pragma unroll
        for (int k = 0; k < K - 1; ++k) v = __builtin_fmaf(a.conv.weight[c * K + k], io::ld(W + k * a.conv.C), v);
        v = __builtin_fmaf(a.conv.weight[c * K + K - 1], io::ld(static_cast<const Tin*>(a.conv.x) + b * a.conv.x_batch + c), v);
        v = silu_scaled(v, 1.0f);
        (i < N ? Bs[i] : i < 2 * N ? Cs[i - N] : xs[i - 2 * N]) = v;
    }
    const float dt = io::ld(static_cast<const Tin*>(a.dt) + b * a.dt_batch + h);
    const float w = softplus_log2(((a.dt_bias ? a.dt_bias[h] : 0.0f) + dt) * kLog2e);
    const float decay = fast_exp2(w * a.A[h]), step = w * kLn2, D = a.D ? a.D[h] : 0.0f;
    __syncthreads();
    float B[E], C[E];
#pragma unroll
    for (int e = 0; e < E; e += 4) {
        io::ld4(Bs + q * E + e, B + e);
        io::ld4(Cs + q * E + e, C + e);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = r * kRows + row;
        const bool live = p0 + i < a.P;
        const float x = xs[live ? i : 0], dx = step * x;
        float y = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s[r][e] = __builtin_fmaf(decay, s[r][e], dx * B[e]);
            y = __builtin_fmaf(C[e], s[r][e], y);
        }
        if (live) {
#pragma unroll
            for (int e = 0; e < E; e += 4) io::st4(S + (int64_t)i * N + e, s[r] + e);
        }
#pragma unroll
        for (int o = 1; o < Q; o <<= 1) y += __shfl_xor(y, o, 64);
        if (live && q == 0) io::st(static_cast<Tout*>(a.y) + bh * a.P + p0 + i, __builtin_fmaf(D, x, y));
    }
}

template <typename Tin, typename Tout, int K, int N, int R>
void launch_r(const M2ConvArgs& a, hipStream_t stream) {
    constexpr int rows = R * kT / (N / (N >= 64 ? 8 : 4));
    KTime kt("m2_conv_step", stream);
    hipLaunchKernelGGL((m2_conv_step_kernel<Tin, Tout, K, N, R>), io::groups(a.batch * a.H * ((a.P + rows - 1) / rows)),
                       dim3(kT), 0, stream, a);
}

template <typename Tin, typename Tout, int K, int N>
hipError_t launch_n(const M2ConvArgs& a, hipStream_t stream) {
    // One row a lane group where a GPU full of workgroups is not there, four
    // where it is: B and C are then made a quarter as often.  us a call, one /
    // four, 32 heads of 64 x 128: batch 1 7.0 / 8.1, 4 7.8 / 8.4, 8 10.0 / 9.6,
    // 32 19.7 / 18.3.
    if (a.batch * a.H * a.P * N < (int64_t)1 << 21) launch_r<Tin, Tout, K, N, 1>(a, stream);
    else launch_r<Tin, Tout, K, N, 4>(a, stream);
    return hipGetLastError();
}

template <typename Tin, typename Tout, int K>
hipError_t by_n(const M2ConvArgs& a, hipStream_t stream) {
    switch (a.N) {
        case 16: return launch_n<Tin, Tout, K, 16>(a, stream);
        case 32: return launch_n<Tin, Tout, K, 32>(a, stream);
        case 64: return launch_n<Tin, Tout, K, 64>(a, stream);
        default: return launch_n<Tin, Tout, K, 128>(a, stream);
    }
}

template <typename Tin, typename Tout>
hipError_t by_k(const M2ConvArgs& a, hipStream_t stream) {
    return a.conv.K == 2 ? by_n<Tin, Tout, 2>(a, stream) : a.conv.K == 3 ? by_n<Tin, Tout, 3>(a, stream) : by_n<Tin, Tout, 4>(a, stream);
}

}  // namespace

hipError_t launch_m2_conv_step(const M2ConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream) {
    hipError_t e;
    if (in_bf16) e = out_bf16 ? by_k<uint16_t, uint16_t>(a, stream) : by_k<uint16_t, float>(a, stream);
    else e = out_bf16 ? by_k<float, uint16_t>(a, stream) : by_k<float, float>(a, stream);
    if (e != hipSuccess) return e;
    return launch_short_conv_step(a.conv, in_bf16, in_bf16, stream);   // (no y: the state alone)
}

}  // namespace selscan
