// m2_conv_rec.hip -- the Mamba-2 mixer token by token, for gfx950.
//
//   S_t = exp(D_t A) S_{t-1} + D_t x_t B_t^T;   y_t = S_t C_t + D x_t
//
// from the convolution's results in fp32 (short_conv.hip, in the workspace).  A
// workgroup has some rows of one head's state in registers, 8 (N >= 64) or 4
// states a lane, and walks the sequence; a row's lanes add y up by shuffles.
// For short sequences: time goes with the length, 0.6 us a token (a chain of
// loads, exponentials and updates) as long as a compute unit has one or two
// workgroups, up to 256 heads of 64 x 128, and with the heads from there (2048:
// 9 us a token).  What both forms take at which lengths stands at kRecTokens in
// mixer.cpp.
#include "io.hpp"
#include "kernels.hpp"

namespace selscan {

namespace {

constexpr int kT = 256;

template <typename Tin, typename Tout, int N>
__global__ __launch_bounds__(kT) void m2_conv_rec_kernel(M2ConvArgs a, const float* X, const float* B, const float* C) {
    constexpr int E = N >= 64 ? 8 : 4, Q = N / E, kRows = kT / Q;
    const int64_t pblocks = (a.P + kRows - 1) / kRows;
    const int64_t id = io::group_id(), bh = id / pblocks;
    if (bh >= a.batch * a.H) return;
    const int64_t b = bh / a.H, h = bh - b * a.H, g = h / (a.H / a.G);
    const int q = threadIdx.x % Q;
    const int64_t pr = (id - bh * pblocks) * kRows + threadIdx.x / Q;
    const bool live = pr < a.P;
    const int64_t p = live ? pr : a.P - 1;
    const int64_t len = a.conv.lengths ? min((int64_t)max(a.conv.lengths[b], 0), a.L) : a.L;
    const float* Xp = X + (b * a.L * a.H + h) * a.P + p;
    const float* Bp = B + (b * a.L * a.G + g) * N + q * E;
    const float* Cp = C + (b * a.L * a.G + g) * N + q * E;
    const Tin* T = static_cast<const Tin*>(a.dt) + b * a.dt_batch + h;
    Tout* Y = static_cast<Tout*>(a.y) + (b * a.L * a.H + h) * a.P + p;
    const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f, D = a.D ? a.D[h] : 0.0f;
    float s[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = a.h0 ? a.h0[(bh * a.P + p) * N + q * E + e] : 0.0f;
    for (int64_t t = 0; t < len; ++t) {
        float bv[E], cv[E];
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            io::Piece<float, 4> pb, pc;   // (not on 16 bytes where H P is odd)
            pb.get(Bp + t * a.G * N + e);
            pc.get(Cp + t * a.G * N + e);
            pb.widen(bv + e);
            pc.widen(cv + e);
        }
        const float x = Xp[t * a.H * a.P];
        const float w = softplus_log2((io::ld(T + t * a.dt_row) + bias) * kLog2e);
        const float decay = fast_exp2(w * A), dx = w * kLn2 * x;
        float y = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s[e] = __builtin_fmaf(decay, s[e], dx * bv[e]);
            y = __builtin_fmaf(cv[e], s[e], y);
        }
#pragma unroll
        for (int o = 1; o < Q; o <<= 1) y += __shfl_xor(y, o, 64);
        if (live && q == 0) io::st(Y + t * a.H * a.P, __builtin_fmaf(D, x, y));
    }
    if (live && q == 0)
        for (int64_t t = len; t < a.L; ++t) io::st(Y + t * a.H * a.P, 0.0f);
    if (a.last && live) {
#pragma unroll
        for (int e = 0; e < E; ++e) a.last[(bh * a.P + p) * N + q * E + e] = s[e];
    }
}

template <typename Tin, typename Tout, int N>
hipError_t launch_n(const M2ConvArgs& a, const float* X, const float* B, const float* C, hipStream_t stream) {
    constexpr int rows = kT / (N / (N >= 64 ? 8 : 4));
    KTime kt("m2_conv_rec", stream);
    hipLaunchKernelGGL((m2_conv_rec_kernel<Tin, Tout, N>), io::groups(a.batch * a.H * ((a.P + rows - 1) / rows)), dim3(kT), 0,
                       stream, a, X, B, C);
    return hipGetLastError();
}

template <typename Tin, typename Tout>
hipError_t by_n(const M2ConvArgs& a, const float* X, const float* B, const float* C, hipStream_t st) {
    switch (a.N) {
        case 16: return launch_n<Tin, Tout, 16>(a, X, B, C, st);
        case 32: return launch_n<Tin, Tout, 32>(a, X, B, C, st);
        case 64: return launch_n<Tin, Tout, 64>(a, X, B, C, st);
        default: return launch_n<Tin, Tout, 128>(a, X, B, C, st);
    }
}

}  // namespace

size_t m2_rec_bytes(const M2ConvArgs& a) { return ((size_t)(a.batch * a.L * a.conv.C) * 4 + 255) & ~size_t(255); }

hipError_t launch_m2_rec(const M2ConvArgs& a, int in_bf16, int out_bf16, void* ws, hipStream_t stream) {
    ShortConvArgs c = a.conv;
    const int64_t rows = a.batch * a.L;
    float* X = static_cast<float*>(ws);
    float* B = X + rows * a.H * a.P;
    float* C = B + rows * a.G * a.N;
    c.y[0] = X; c.y[1] = B; c.y[2] = C;
    const hipError_t e = launch_short_conv_fwd(c, in_bf16, 0, stream);
    if (e != hipSuccess) return e;
    if (in_bf16) return out_bf16 ? by_n<uint16_t, uint16_t>(a, X, B, C, stream) : by_n<uint16_t, float>(a, X, B, C, stream);
    return out_bf16 ? by_n<float, uint16_t>(a, X, B, C, stream) : by_n<float, float>(a, X, B, C, stream);
}

}  // namespace selscan
