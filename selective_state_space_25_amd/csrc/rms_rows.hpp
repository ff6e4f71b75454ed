// rms_rows.hpp -- what the RMS norm's two directions share: how a row's group
// lies on the lanes, loads and stores of its pieces, sums over it.
#pragma once

#include "io.hpp"
#include "kernels.hpp"

namespace selscan {
namespace rms {

constexpr int kT = 256;
constexpr int kLongest = 8192;   // elements of a group that stay in registers

// Up to eight elements (n of them, the others zero) at any element's address.
// FULL: n >= 8 is known.
template <bool FULL, typename T>
__device__ __forceinline__ void ldp(const T* p, int n, float (&v)[8]) {
    if (FULL || n >= 8) {
        io::Piece<T, 8> r;
        r.get(p);
        r.widen(v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? io::ld(p + i) : 0.0f;
    }
}
template <bool FULL, typename T>
__device__ __forceinline__ void stp(T* p, int n, const float (&v)[8]) {
    if (FULL || n >= 8) {
        io::Piece<T, 8> r;
        r.narrow(v);
        r.put(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) io::st(p + i, v[i]);
    }
}
// e4m3 (round to nearest even), which no value here is past.
template <bool FULL>
__device__ __forceinline__ void stp(uint8_t* p, int n, const float (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], q, true);
    }
    struct __attribute__((packed, may_alias, aligned(1))) Loose { uint32_t a, b; };
    if (FULL || n >= 8) {
        *reinterpret_cast<Loose*>(p) = {w[0], w[1]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// Sum, and largest, over the LR lanes that hold a group, the same value in
// each of them.  LR = 256: the workgroup; else an aligned part of a wave.
template <int LR, typename T, typename F>
__device__ __forceinline__ T over_row(T v, T* sm, F f) {
#pragma unroll
    for (int o = (LR < 64 ? LR : 64) / 2; o >= 1; o >>= 1) v = f(v, (T)__shfl_xor(v, o, 64));
    if constexpr (LR == 256) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
        __syncthreads();
        v = f(f(sm[0], sm[1]), f(sm[2], sm[3]));
    }
    return v;
}
template <int LR>
__device__ __forceinline__ float row_sum(float v, float* sm) {
    return over_row<LR>(v, sm, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ float sigmoid(float z) { return fast_rcp(1.0f + fast_exp2(-z * kLog2e)); }

// Lanes a group takes and pieces a lane (0: the group is too long).  A group of
// up to `wave` pieces stays in one wave, a longer one takes the four of a
// workgroup: more loads in flight a group, but barriers, and idle lanes where
// its pieces are not a multiple of 256 by far.
struct Layout {
    int lanes, pieces;
    Layout(int64_t width, int wave) {
        const int64_t np = (width + 7) / 8;
        lanes = np <= 8 ? 8 : np <= 16 ? 16 : np <= 32 ? 32 : np <= wave ? 64 : 256;
        pieces = width > kLongest ? 0 : (int)((np + lanes - 1) / lanes);
    }
    int at_once() const { return pieces ? kT / lanes : 1; }   // groups a workgroup has at a time
};

// f.template run<LR, NV>() of the layout, whose `wave` lies between 64 (LEAST -
// 1) and 64 MOST pieces.
template <int LEAST, int MOST, typename F>
hipError_t by_layout(const Layout& l, F f) {
    if (l.lanes == 8) return f.template run<8, 1>();
    if (l.lanes == 16) return f.template run<16, 1>();
    if (l.lanes == 32) return f.template run<32, 1>();
    if (l.lanes == 256) {
        if constexpr (LEAST <= 4) {
            if (l.pieces == 1) return f.template run<256, 1>();
        }
        return l.pieces == 2 ? f.template run<256, 2>() : l.pieces == 3 ? f.template run<256, 3>() : f.template run<256, 4>();
    }
    if constexpr (MOST >= 4) {
        if (l.pieces == 4) return f.template run<64, 4>();
        if (l.pieces == 5) return f.template run<64, 5>();
    }
    return l.pieces == 1 ? f.template run<64, 1>() : l.pieces == 2 ? f.template run<64, 2>() : f.template run<64, 3>();
}

}  // namespace rms
}  // namespace selscan
