// delta_rec.hip -- the gated delta rule token by token (fp32 state in
// registers): one decoded token, updated in place, and short sequences.
//
// Row p of a head's state [P, N] meets its own v_p and y_p and the head's q
// and k, so rows are independent.  With a = exp(g), per row and token
//
//   u = beta (v - a S.k);   y = scale (a S.q + u k.q);   S = a S + u k
//
// where S.k, S.q and k.q are sums over the row's old state, reduced together
// across the Q lanes that share a row: one reduction a token, not two.
//
// One token is bound by the state's bytes: batch 128, 16 heads of 128 x 128,
// 270 MB read and written in 51 to 53 us over one state again and again (5.2
// TB/s, what a copy reaches), 63 us over two in turn, which no cache holds a
// part of.  A single small sequence (32 heads of 64 x 128) is the launch: 4.3
// us a call bound, 9.5 unbound.
#include "io.hpp"
#include "kernels.hpp"

namespace selscan {

namespace {

template <int Q>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = 1; o < Q; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// Q lanes per row, E states per lane in 4-element pieces: piece j of lane i
// starts at state 4 (i + Q j).
template <typename Tin, typename Tout, int Q, int E>
__global__ __launch_bounds__(256) void delta_rec_kernel(DeltaArgs a) {
    const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t rows = a.batch * a.H * a.P;
    const int64_t row_raw = gid / Q;
    const bool ok = row_raw < rows;
    const int64_t row = ok ? row_raw : rows - 1;
    const int qi = (int)(gid % Q);
    const int64_t bh = row / a.P;
    const int64_t p = row - bh * a.P;
    const int64_t b = bh / a.H;
    const int64_t h = bh - b * a.H;
    const int64_t grp = h / (a.H / a.G);
    const int N = a.N;
    const int64_t len = a.lengths ? min((int64_t)max(a.lengths[b], 0), a.L) : a.L;

    float s[E];
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
        const int n = 4 * (qi + Q * j);
        if (!a.h0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * j + i] = 0.0f;
        } else if (a.vec) {
            if (n < N) {
                io::ld4(a.h0 + row * N + n, s + 4 * j);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[4 * j + i] = 0.0f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * j + i] = n + i < N ? a.h0[row * N + n + i] : 0.0f;
        }
    }
    for (int64_t t = 0; t < len; ++t) {
        const int64_t bt = b * a.L + t;
        const Tin* qp = reinterpret_cast<const Tin*>(a.q) + (bt * a.G + grp) * N;
        const Tin* kp = reinterpret_cast<const Tin*>(a.k) + (bt * a.G + grp) * N;
        float q[E], k[E];
#pragma unroll
        for (int j = 0; j < E / 4; ++j) {
            const int n = 4 * (qi + Q * j);
            if (a.vec && n < N) {
                io::ld4(qp + n, q + 4 * j);
                io::ld4(kp + n, k + 4 * j);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    q[4 * j + i] = n + i < N ? io::ld(qp + n + i) : 0.0f;
                    k[4 * j + i] = n + i < N ? io::ld(kp + n + i) : 0.0f;
                }
            }
        }
        const float v = io::ld(reinterpret_cast<const Tin*>(a.v) + (bt * a.H + h) * a.P + p);
        const float dec = fast_exp2(a.g[bt * a.H + h] * kLog2e);
        const float beta = a.beta[bt * a.H + h];
        float sk = 0.0f, sq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sk = __builtin_fmaf(s[e], k[e], sk);
            sq = __builtin_fmaf(s[e], q[e], sq);
            kq = __builtin_fmaf(k[e], q[e], kq);
        }
        sk = group_sum<Q>(sk);
        sq = group_sum<Q>(sq);
        kq = group_sum<Q>(kq);
        const float u = beta * __builtin_fmaf(-dec, sk, v);
        const float y = a.scale * __builtin_fmaf(u, kq, dec * sq);
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] = __builtin_fmaf(u, k[e], dec * s[e]);
        if (ok && qi == 0) io::st(reinterpret_cast<Tout*>(a.y) + (bt * a.H + h) * a.P + p, y);
    }
    for (int64_t t = len; t < a.L; ++t)
        if (ok && qi == 0) io::st(reinterpret_cast<Tout*>(a.y) + ((b * a.L + t) * a.H + h) * a.P + p, 0.0f);
    if (!ok || !a.last) return;
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
        const int n = 4 * (qi + Q * j);
        if (a.vec && n < N) {
            io::st4(a.last + row * N + n, s + 4 * j);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < N) a.last[row * N + n + i] = s[4 * j + i];
        }
    }
}

template <typename Tin, typename Tout, int Q, int E>
hipError_t launch(const DeltaArgs& a, hipStream_t stream) {
    const int64_t threads = a.batch * a.H * a.P * Q;
    KTime kt("delta_rec", stream);
    hipLaunchKernelGGL((delta_rec_kernel<Tin, Tout, Q, E>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0,
                       stream, a);
    return hipGetLastError();
}

template <typename Tin, typename Tout>
hipError_t by_n(const DeltaArgs& a, hipStream_t stream) {
    if (a.N <= 16) return launch<Tin, Tout, 4, 4>(a, stream);
    if (a.N <= 32) return launch<Tin, Tout, 8, 4>(a, stream);
    if (a.N <= 64) return launch<Tin, Tout, 16, 4>(a, stream);
    return launch<Tin, Tout, 16, 8>(a, stream);
}

}  // namespace

hipError_t launch_delta_rec(const DeltaArgs& a, int in_bf16, int out_bf16, hipStream_t stream) {
    if (in_bf16) return out_bf16 ? by_n<uint16_t, uint16_t>(a, stream) : by_n<uint16_t, float>(a, stream);
    return out_bf16 ? by_n<float, uint16_t>(a, stream) : by_n<float, float>(a, stream);
}

}  // namespace selscan
