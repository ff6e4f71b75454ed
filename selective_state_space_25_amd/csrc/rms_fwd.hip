// rms_fwd.hip -- RMS norm with what stands in front of it, for gfx950.
//
//   s = x + residual, or x silu(gate);  rstd = 1 / sqrt(sum s^2 / width + eps);  y = s rstd weight
//
// over the groups of a row (one group: the row), y in fp32, bf16 or, with a
// scale for each block of a group, e4m3: scale = max(max |y| / 448, 2^-126), the
// fp32 quotient y / scale rounded to nearest even.  A stream bound by memory: a
// group stays in registers between its sum and its output, in 8-element pieces
// over 8 to 64 lanes of a wave (up to 1024 to 1536 elements, sums without a
// barrier) or the 256 of a workgroup (to 8192), so every element is read once
// and written once; the 8-bit form costs a shuffle of a block's lanes and no
// second pass.  Narrow groups share a wave.  Rows may start at any element's
// address and end inside a piece.  Longer groups are read again for each step.
//
// 32768 x 2560, bf16 with an fp32 residual: 182 us for 1.01 GB, 5.5 TB/s.
// 16384 x 5120 with a gate, e4m3 in blocks of 128: 102 us for 0.42 GB, 4.1 TB/s,
// vector ALU 80 % busy (silu, the blocks' maxima, quotients, conversions).  One
// row of 768 is the launch: 2.8 us.
#include "rms_rows.hpp"

namespace selscan {

namespace {

using namespace rms;

constexpr float kTop8 = 448.0f;
constexpr float kLeastScale = 1.1754943508222875e-38f;   // 2^-126

// The elements' absolute values as integers: a NaN is larger than any number.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ float scale_of(uint32_t m) {
    const float s = __uint_as_float(m) / kTop8;
    return s < kLeastScale ? kLeastScale : s;   // (NaN stays)
}

// v / scale, rounded as a division is: a product with the rounded reciprocal is
// off in one of four quotients, and next to a tie of e4m3 that costs a whole
// step.  One correction from the exact remainder makes it the division's
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) where nothing leaves fp32's range; scales outside 2^-80 ..
// 2^100 (NaN among them) are divided by.
__device__ __forceinline__ void over_scale(float (&v)[8], float scale, float inv) {
    if (scale >= 0x1p-80f && scale <= 0x1p100f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = v[i] * inv;
            v[i] = __builtin_fmaf(__builtin_fmaf(-q, scale, v[i]), inv, q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] /= scale;
    }
}

// One group of one row.
template <typename Tin, typename Tres, typename Tout>
struct Row {
    const Tin *x, *z;
    const Tres* r;
    const float* w;
    Tout* y;
    Tres* s;
    float* scale;
    int width;
    __device__ __forceinline__ Row(const RmsArgs& a, int64_t unit) {
        const int64_t base = unit * a.width, row = a.groups == 1 ? unit : unit / a.groups;
        const int64_t g0 = (unit - row * a.groups) * a.width;
        x = static_cast<const Tin*>(a.x) + base;
        z = a.gate ? static_cast<const Tin*>(a.gate) + row * a.gate_row + g0 : nullptr;
        r = a.res ? static_cast<const Tres*>(a.res) + base : nullptr;
        w = a.weight ? a.weight + g0 : nullptr;
        y = static_cast<Tout*>(a.y) + base;
        s = a.res_out ? static_cast<Tres*>(a.res_out) + base : nullptr;
        scale = a.scale ? a.scale + unit * a.row_blocks : nullptr;
        width = (int)a.width;
    }
    // s of the piece from element d
    template <bool FULL>
    __device__ __forceinline__ void sum(int d, float (&v)[8]) const {
        float t[8];
        ldp<FULL>(x + d, width - d, v);
        if (z) {
            ldp<FULL>(z + d, width - d, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= silu_scaled(t[i], 1.0f);
        }
        if (r) {
            ldp<FULL>(r + d, width - d, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += t[i];
        }
    }
    // y of the piece from its s
    template <bool FULL>
    __device__ __forceinline__ void norm(int d, float rstd, float (&v)[8]) const {
        float t[8];
        if (w) ldp<FULL>(w + d, width - d, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] *= rstd;
            if (w) v[i] *= t[i];
        }
    }
};

template <typename Tin, typename Tres, typename Tout, int LR, int NV>
__global__ __launch_bounds__(kT) void rms_fwd_kernel(RmsArgs a) {
    __shared__ float sm[4];
    constexpr bool k8 = sizeof(Tout) == 1;
    const int at = threadIdx.x % LR;
    const int64_t unit = io::group_id() * (kT / LR) + threadIdx.x / LR;
    if (unit >= a.rows * a.groups) return;   // (all lanes of a group together)
    const Row<Tin, Tres, Tout> row(a, unit);
    float s[NV][8];
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int d = 8 * (at + LR * j);
        if (j + 1 < NV) row.template sum<true>(d, s[j]);
        else if (d < row.width) row.template sum<false>(d, s[j]);
        else {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] = 0.0f;
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
    #pragma unroll
        for (int i = 0; i < 8; ++i) sq = __builtin_fmaf(s[j][i], s[j][i], sq);
    }
    const float rstd = 1.0f / sqrtf(row_sum<LR>(sq, sm) * a.inv_width + a.eps);
    if (at == 0 && a.rstd) a.rstd[unit] = rstd;
    uint32_t top = 0;
    const int block = (int)a.block, shift = __builtin_ctz(block | (1 << 30));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int d = 8 * (at + LR * j);
        auto piece = [&](auto full) {
            constexpr bool FULL = decltype(full)::value;
            if (row.s) stp<FULL>(row.s + d, row.width - d, s[j]);
            row.template norm<FULL>(d, rstd, s[j]);
            if constexpr (!k8) stp<FULL>(row.y + d, row.width - d, s[j]);
        };
        if (j + 1 < NV) piece(std::true_type());
        else if (d < row.width) piece(std::false_type());
        if constexpr (k8) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = larger(m, magnitude(s[j][i]));
            if (block) {
                // a block is 4 to 64 lanes of a wave; narrower groups are one block
                for (int o = min(block / 8, LR) / 2; o >= 1; o >>= 1) m = larger(m, (uint32_t)__shfl_xor((int)m, o, 64));
                const float sc = scale_of(m);
                over_scale(s[j], sc, 1.0f / sc);
                if (d < row.width) {
                    if ((d & (block - 1)) == 0) row.scale[d >> shift] = sc;
                    stp<false>(row.y + d, row.width - d, s[j]);
                }
            } else {
                top = larger(top, m);
            }
        }
    }
    if constexpr (k8) {
        if (a.block) return;
        __shared__ uint32_t sm8[4];
        const float sc = scale_of(over_row<LR>(top, sm8, larger)), inv = 1.0f / sc;
        if (at == 0) row.scale[0] = sc;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = 8 * (at + LR * j);
            over_scale(s[j], sc, inv);
            if (d < row.width) stp<false>(row.y + d, row.width - d, s[j]);
        }
    }
}

// Groups longer than the registers: read again for each step, 2048 elements at
// a time.  A lane's sum over those is fp64: in fp32 its error grows with the
// length, as fast as that where the terms are alike.
template <typename Tin, typename Tres, typename Tout>
__global__ __launch_bounds__(kT) void rms_fwd_long_kernel(RmsArgs a) {
    __shared__ float sm[4];
    __shared__ uint32_t sm8[4];
    constexpr bool k8 = sizeof(Tout) == 1;
    const int64_t unit = io::group_id();
    if (unit >= a.rows * a.groups) return;
    const Row<Tin, Tres, Tout> row(a, unit);
    float v[8];
    double sq = 0.0;
    for (int d = 8 * (int)threadIdx.x; d < row.width; d += 8 * kT) {
        float p = 0.0f;
        row.template sum<false>(d, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) p = __builtin_fmaf(v[i], v[i], p);
        sq += p;
    }
    const float rstd = 1.0f / sqrtf(row_sum<256>((float)sq, sm) * a.inv_width + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[unit] = rstd;
    float sc = 1.0f, inv = 1.0f;
    if constexpr (k8) {
        if (!a.block) {
            uint32_t m = 0;
            for (int d = 8 * (int)threadIdx.x; d < row.width; d += 8 * kT) {
                row.template sum<false>(d, v);
                row.template norm<false>(d, rstd, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) m = larger(m, magnitude(v[i]));
            }
            sc = scale_of(over_row<256>(m, sm8, larger));
            inv = 1.0f / sc;
            if (threadIdx.x == 0) row.scale[0] = sc;
        }
    }
    for (int d0 = 0; d0 < row.width; d0 += 8 * kT) {   // (all lanes take every turn: blocks are shuffled)
        const int d = d0 + 8 * (int)threadIdx.x;
        const bool live = d < row.width;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (live) {
            row.template sum<false>(d, v);
            if (row.s) stp<false>(row.s + d, row.width - d, v);
            row.template norm<false>(d, rstd, v);
        }
        if constexpr (k8) {
            if (a.block) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = larger(m, magnitude(v[i]));
                for (int o = (int)(a.block / 16); o >= 1; o >>= 1) m = larger(m, (uint32_t)__shfl_xor((int)m, o, 64));
                sc = scale_of(m);
                inv = 1.0f / sc;
                if (live && d % a.block == 0) row.scale[d / a.block] = sc;
            }
            over_scale(v, sc, inv);
        }
        if (live) stp<false>(row.y + d, row.width - d, v);
    }
}

template <typename Tin, typename Tres, typename Tout>
struct Fwd {
    const RmsArgs& a;
    hipStream_t stream;
    template <int LR, int NV>
    hipError_t run() {
        KTime kt("rms_fwd", stream);
        constexpr int n = kT / LR;
        hipLaunchKernelGGL((rms_fwd_kernel<Tin, Tres, Tout, LR, NV>), io::groups((a.rows * a.groups + n - 1) / n), dim3(kT),
                           0, stream, a);
        return hipGetLastError();
    }
};

// Pieces of a group that stay in one wave: fewer where an element moves more
// bytes (a residual counts with its s, asked for or not: y has the same bits).
// us, one wave / four, 2^26 elements (bf16 unless it says fp32):
//   bytes              1088         1280         1536         1664         2048         2560
//   4  x, y           54 /  81     50 /  70     48 /  60     52 /  59     51 /  51     51 /  54
//   5  gate, e4m3     96 / 132     86 / 115     75 /  95     93 /  94     80 /  78     90 /  91
//   6  gate           82 / 111     78 /  98     77 /  85     83 /  84     84 /  74     84 /  82
//   6  fp32 x         71 /  84     71 /  77     71 /  71     73 /  71     72 /  68     74 /  70
//   8  residual, s   103 / 119    103 / 105    104 /  96    110 /  95    108 /  92    109 /  98
//   8  fp32 x, y     101 / 101    103 / 101    102 /  97    104 /  98    105 /  94    107 /  98
//   8  gate, fp32 y  111 / 125    111 / 113    110 / 106    117 / 106    116 / 100    118 / 109
//   12 fp32 residual 155 / 145    159 / 147    158 / 143    164 / 143    167 / 140    167 / 147
//   12 gate, fp32    146 / 142    149 / 143    150 / 139    152 / 140    152 / 138    157 / 142
template <typename Tin, typename Tres, typename Tout>
int wave_pieces(const RmsArgs& a) {
    const int bytes = (int)sizeof(Tin) * (a.gate ? 2 : 1) + (int)sizeof(Tres) * (a.res ? 2 : 0) + (int)sizeof(Tout);
    return bytes > 8 ? 128 : bytes == 8 ? 160 : 192;
}

template <typename Tin, typename Tres, typename Tout>
hipError_t fwd(const RmsArgs& a, hipStream_t stream) {
    const Layout l(a.width, wave_pieces<Tin, Tres, Tout>(a));
    if (l.pieces) return by_layout<3, 3>(l, Fwd<Tin, Tres, Tout>{a, stream});
    KTime kt("rms_fwd", stream);
    hipLaunchKernelGGL((rms_fwd_long_kernel<Tin, Tres, Tout>), io::groups(a.rows * a.groups), dim3(kT), 0, stream, a);
    return hipGetLastError();
}

template <typename Tin, typename Tres>
hipError_t by_out(const RmsArgs& a, int out_dtype, hipStream_t st) {
    return out_dtype == SELSCAN_E4M3 ? fwd<Tin, Tres, uint8_t>(a, st)
           : out_dtype == SELSCAN_BF16 ? fwd<Tin, Tres, uint16_t>(a, st) : fwd<Tin, Tres, float>(a, st);
}

}  // namespace

hipError_t launch_rms_fwd(const RmsArgs& a, int in_bf16, int res_bf16, int out_dtype, hipStream_t stream) {
    if (in_bf16) return res_bf16 ? by_out<uint16_t, uint16_t>(a, out_dtype, stream) : by_out<uint16_t, float>(a, out_dtype, stream);
    return res_bf16 ? by_out<float, uint16_t>(a, out_dtype, stream) : by_out<float, float>(a, out_dtype, stream);
}

}  // namespace selscan
