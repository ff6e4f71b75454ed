// norm.hip -- layer norm with the dropout and the residual sum in front of
// it, forward and gradients.
//
//   s = dropout(x) + residual;  y = (s - mean) rstd weight + bias
//   ds = rstd (w - mean_d w - xhat mean_d (w xhat)) + dresidual,  w = dy weight
//   dweight = sum_r dy xhat;  dbias = sum_r dy
//
// Both directions are streams bound by memory.  A row stays in registers
// between its sums and its output: 8-element pieces over the 64 lanes of one
// wave (rows to 2560 elements, sums without a barrier) or the 256 of a
// workgroup (to 8192); longer rows, and rows that are not made of aligned
// 16-byte pieces, are read again for each step instead.  The variance is
// summed over (s - mean)^2, not taken as a difference of moments.  The
// gradients' waves walk rows a fixed distance apart and keep their sums for
// dweight and dbias in registers, one partial row a workgroup, which a second
// kernel adds in a fixed order.  A wave adds up 64 rows at most (there are
// more workgroups where there are more rows), the second kernel in fp64: a
// plain fp32 sum of all that a wave would get, thousands of short rows, is off
// by 1e-4 where its roundings lean one way.
//
// Measured at 32768 rows, bf16 x and y, fp32 residual, dropout 0.1:
//
//   dim    forward                  gradients
//   2560   207 us (4.9 TB/s)        263 us (5.1 TB/s)
//   4096   300 us (5.4 TB/s)        417 us (5.2 TB/s)
//   2557   763 us                   553 us (417, 128 for dweight and dbias, 8)
//
// The last reads rows again: scalar loads, three passes in either direction,
// and in the forward one ten-round generator call for each element and pass
// (vector ALU 74 % busy).  One row of 768 is the launch: 16 us a call, 6 of
// them the kernel's.
#include <algorithm>

#include "io.hpp"
#include "kernels.hpp"
#include "philox.hpp"

namespace selscan {

namespace {

constexpr int kT = 256;

// Sum over the workgroup, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
    __syncthreads();
    return (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

// The pieces' values after dropout: base: index of the first element.
__device__ __forceinline__ void drop8(const NormArgs& a, int64_t base, float* v) {
    uint32_t w[8];
    philox4((uint64_t)base >> 2, a.offset, a.seed, w);
    philox4(((uint64_t)base >> 2) + 1, a.offset, a.seed, w + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i] >= a.keep_from ? v[i] * a.keep_scale : 0.0f;
}

// Sum over the row's W waves, the same value in every lane.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* sm) {
    if constexpr (W == 4) return block_sum(v, sm);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// W waves per row (a workgroup has 4 / W rows), NV pieces per lane.
template <typename Tin, typename Tres, typename Tout, int W, int NV>
__global__ __launch_bounds__(kT) void norm_fwd_reg_kernel(NormArgs a) {
    __shared__ float sm[4];
    const int at = threadIdx.x % (64 * W);
    const int64_t row = io::group_id() * (4 / W) + threadIdx.x / (64 * W);
    if (row >= a.rows) return;   // (a wave's row is its own when W is 1, the workgroup's when W is 4)
    const int64_t base = row * a.dim;
    const Tin* X = reinterpret_cast<const Tin*>(a.x) + base;
    const Tres* R = a.res ? reinterpret_cast<const Tres*>(a.res) + base : nullptr;
    const int np = (int)(a.dim / 8);
    float s[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int d = 8 * (at + 64 * W * j);
        if (at + 64 * W * j < np) {
            float r[8];
            io::ld8(X + d, s[j]);
            if (R) io::ld8(R + d, r);
            if (a.drop) drop8(a, base + d, s[j]);
            if (R) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[j][i] += r[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += s[j][i];
        }
    }
    const float mean = row_sum<W>(sum, sm) * a.inv_dim;
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (at + 64 * W * j < np) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sq = __builtin_fmaf(s[j][i] - mean, s[j][i] - mean, sq);
        }
    const float rstd = 1.0f / sqrtf(row_sum<W>(sq, sm) * a.inv_dim + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int d = 8 * (at + 64 * W * j);
        if (at + 64 * W * j >= np) continue;
        if (a.res_out) io::st8(reinterpret_cast<Tres*>(a.res_out) + base + d, s[j]);
        float w[8], b[8];
        if (a.weight) io::ld8(a.weight + d, w);
        if (a.bias) io::ld8(a.bias + d, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y = (s[j][i] - mean) * rstd;
            if (a.weight) y *= w[i];
            if (a.bias) y += b[i];
            s[j][i] = y;
        }
        io::st8(reinterpret_cast<Tout*>(a.y) + base + d, s[j]);
    }
    if (at == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

template <typename Tin, typename Tres, typename Tout, int W, int NV>
__global__ __launch_bounds__(kT) void norm_bwd_reg_kernel(NormArgs a) {
    __shared__ float sm[4];
    __shared__ float part[W == 1 ? 4 * 512 : 1];
    const int at = threadIdx.x % (64 * W), np = (int)(a.dim / 8);
    float gw[NV][8], gb[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) gw[j][i] = gb[j][i] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.x * (4 / W) + threadIdx.x / (64 * W); row < a.rows; row += (int64_t)gridDim.x * (4 / W)) {
        const int64_t base = row * a.dim;
        const Tout* DY = reinterpret_cast<const Tout*>(a.x) + base;
        const Tres* S = reinterpret_cast<const Tres*>(a.res) + base;
        const Tres* DR = a.dres_in ? reinterpret_cast<const Tres*>(a.dres_in) + base : nullptr;
        const float mean = a.mean_in[row], rstd = a.rstd_in[row];
        float y[NV][8], x[NV][8];
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = 8 * (at + 64 * W * j);
            if (at + 64 * W * j >= np) continue;
            io::ld8(DY + d, y[j]);
            io::ld8(S + d, x[j]);
            float w[8];
            if (a.weight) io::ld8(a.weight + d, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[j][i] = (x[j][i] - mean) * rstd;
                gw[j][i] = __builtin_fmaf(y[j][i], x[j][i], gw[j][i]);
                gb[j][i] += y[j][i];
                if (a.weight) y[j][i] *= w[i];
                c1 += y[j][i];
                c2 = __builtin_fmaf(y[j][i], x[j][i], c2);
            }
        }
        if (!a.y && !a.res_out) continue;
        c1 = row_sum<W>(c1, sm) * a.inv_dim;
        c2 = row_sum<W>(c2, sm) * a.inv_dim;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = 8 * (at + 64 * W * j);
            if (at + 64 * W * j >= np) continue;
            float r[8];
            if (DR) io::ld8(DR + d, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[j][i] = (y[j][i] - c1 - x[j][i] * c2) * rstd;
                if (DR) y[j][i] += r[i];
            }
            if (a.res_out) io::st8(reinterpret_cast<Tres*>(a.res_out) + base + d, y[j]);
            if (a.y) {
                if (a.drop) drop8(a, base + d, y[j]);
                io::st8(reinterpret_cast<Tin*>(a.y) + base + d, y[j]);
            }
        }
    }
    if (!a.dweight && !a.dbias) return;
    float* out = a.part + 2 * (int64_t)blockIdx.x * a.dim;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float (&v)[8] = g ? gb[j] : gw[j];
            const int d = 8 * (at + 64 * W * j);
            if constexpr (W == 4) {
                if (at + 64 * W * j < np) io::st8(out + g * a.dim + d, v);
            } else {   // the four waves' sums of the same columns, in their order
                __syncthreads();
                io::st8(part + (threadIdx.x >> 6) * 512 + 8 * at, v);
                __syncthreads();
                for (int e = threadIdx.x; e < 512 && 512 * j + e < a.dim; e += kT)
                    out[g * a.dim + 512 * j + e] = ((part[e] + part[512 + e]) + part[1024 + e]) + part[1536 + e];
            }
        }
    }
}

__device__ __forceinline__ float dropped(const NormArgs& a, int64_t i, float v) {
    uint32_t w[4];
    philox4((uint64_t)i >> 2, a.offset, a.seed, w);
    const int k = (int)(i & 3);
    const uint32_t r = k == 0 ? w[0] : k == 1 ? w[1] : k == 2 ? w[2] : w[3];
    return r >= a.keep_from ? v * a.keep_scale : 0.0f;
}

template <typename Tin, typename Tres, typename Tout>
__global__ __launch_bounds__(kT) void norm_fwd_kernel(NormArgs a) {
    __shared__ float sm[4];
    const int64_t row = io::group_id();
    if (row >= a.rows) return;
    const int64_t base = row * a.dim;
    const Tin* X = reinterpret_cast<const Tin*>(a.x) + base;
    const Tres* R = a.res ? reinterpret_cast<const Tres*>(a.res) + base : nullptr;
    auto value = [&](int64_t d) {
        float v = io::ld(X + d);
        if (a.drop) v = dropped(a, base + d, v);
        return R ? v + io::ld(R + d) : v;
    };
    float sum = 0.0f;
    for (int64_t d = threadIdx.x; d < a.dim; d += kT) sum += value(d);
    const float mean = block_sum(sum, sm) * a.inv_dim;
    float sq = 0.0f;
    for (int64_t d = threadIdx.x; d < a.dim; d += kT) {
        const float c = value(d) - mean;
        sq += c * c;
    }
    const float rstd = 1.0f / sqrtf(block_sum(sq, sm) * a.inv_dim + a.eps);
    for (int64_t d = threadIdx.x; d < a.dim; d += kT) {
        const float s = value(d);
        const float n = (s - mean) * rstd * (a.weight ? a.weight[d] : 1.0f) + (a.bias ? a.bias[d] : 0.0f);
        if (a.res_out) io::st(reinterpret_cast<Tres*>(a.res_out) + base + d, s);
        io::st(reinterpret_cast<Tout*>(a.y) + base + d, n);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

template <typename Tin, typename Tres, typename Tout>
__global__ __launch_bounds__(kT) void norm_bwd_kernel(NormArgs a) {
    __shared__ float sm[4];
    const int64_t row = io::group_id();
    if (row >= a.rows) return;
    const int64_t base = row * a.dim;
    const Tout* DY = reinterpret_cast<const Tout*>(a.x) + base;
    const Tres* S = reinterpret_cast<const Tres*>(a.res) + base;
    const Tres* DR = a.dres_in ? reinterpret_cast<const Tres*>(a.dres_in) + base : nullptr;
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t d = threadIdx.x; d < a.dim; d += kT) {
        const float w = io::ld(DY + d) * (a.weight ? a.weight[d] : 1.0f);
        c1 += w;
        c2 += w * ((io::ld(S + d) - mean) * rstd);
    }
    c1 = block_sum(c1, sm) * a.inv_dim;
    c2 = block_sum(c2, sm) * a.inv_dim;
    for (int64_t d = threadIdx.x; d < a.dim; d += kT) {
        const float w = io::ld(DY + d) * (a.weight ? a.weight[d] : 1.0f);
        const float xh = (io::ld(S + d) - mean) * rstd;
        float ds = (w - c1 - xh * c2) * rstd;
        if (DR) ds += io::ld(DR + d);
        if (a.res_out) io::st(reinterpret_cast<Tres*>(a.res_out) + base + d, ds);
        if (a.y) io::st(reinterpret_cast<Tin*>(a.y) + base + d, a.drop ? dropped(a, base + d, ds) : ds);
    }
}

// A sum over rows that keeps what each addition rounds off (Kahan).
struct RowSum {
    float s = 0.0f, c = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float y = v - c, t = s + y;
        c = (t - s) - y;
        s = t;
    }
};

// Partial sums of dweight and dbias: workgroup (x, y) takes 256 columns and
// every gridDim.y-th row, however many those are.
template <typename Tres, typename Tout>
__global__ __launch_bounds__(kT) void norm_wgrad_kernel(NormArgs a) {
    const int64_t d = (int64_t)blockIdx.x * kT + threadIdx.x;
    if (d >= a.dim) return;
    const Tout* DY = reinterpret_cast<const Tout*>(a.x) + d;
    const Tres* S = reinterpret_cast<const Tres*>(a.res) + d;
    RowSum gw, gb;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float dy = io::ld(DY + r * a.dim);
        gw.add(dy * ((io::ld(S + r * a.dim) - a.mean_in[r]) * a.rstd_in[r]));
        gb.add(dy);
    }
    a.part[(2 * (int64_t)blockIdx.y) * a.dim + d] = gw.s;
    a.part[(2 * (int64_t)blockIdx.y + 1) * a.dim + d] = gb.s;
}

// Sums of n partial rows [n, 2, dim]: workgroup (x, y) takes 64 columns and
// kSumRows of the rows, in 16 slices; the sums of y lie 2 dim y further on.
constexpr int kSumRows = 1024;
__global__ __launch_bounds__(1024) void norm_wsum_kernel(const float* part, int n, int64_t dim, float* dweight, float* dbias) {
    __shared__ double sm[2][16][64];
    const int col = threadIdx.x & 63, sl = threadIdx.x >> 6;
    const int64_t d = (int64_t)blockIdx.x * 64 + col;
    const int end = min(n, (int)(blockIdx.y + 1) * kSumRows);
    double gw = 0.0, gb = 0.0;
    if (d < dim) {
#pragma unroll 4
        for (int b = (int)blockIdx.y * kSumRows + sl; b < end; b += 16) {
            gw += part[2 * (int64_t)b * dim + d];
            gb += part[(2 * (int64_t)b + 1) * dim + d];
        }
    }
    sm[0][sl][col] = gw;
    sm[1][sl][col] = gb;
    __syncthreads();
    if (sl < 2 && d < dim) {
        double v = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += sm[sl][i][col];
        float* out = sl ? dbias : dweight;
        if (out) out[2 * (int64_t)blockIdx.y * dim + d] = (float)v;
    }
}

constexpr int kBlocks = 512;

// Rows that a workgroup of the register kernels works on at a time: one wave
// or four to a row.  Past five pieces a lane the gradients' sums no longer fit
// a wave's registers beside the row.  us, one wave / four, 2^26 elements, bf16
// x and y, fp32 residual:
//
//   dim     512          1024         2048         2560         2816
//   fwd     143 / 207    142 / 145    149 / 137    155 / 145    156 / 144
//   grad    200 / 344    192 / 218    196 / 213    206 / 253    295 / 241
//
// One rule serves both directions: it is the gradients', the longer of them.
int rows_at_once(int64_t dim) { return dim / 8 <= 5 * 64 ? 4 : 1; }

// Waves per row and pieces per lane of the register kernels; 0: neither fits.
int reg_pieces(const NormArgs& a, int& waves) {
    if (!a.vec || a.dim > 8192) return 0;
    const int np = (int)(a.dim / 8);
    waves = 4 / rows_at_once(a.dim);
    return (np + 64 * waves - 1) / (64 * waves);
}

template <bool FWD, typename Tin, typename Tres, typename Tout, int W, int NV>
hipError_t reg(const NormArgs& a, hipStream_t stream) {
    KTime kt(FWD ? "norm_fwd" : "norm_bwd", stream);
    if constexpr (FWD)
        hipLaunchKernelGGL((norm_fwd_reg_kernel<Tin, Tres, Tout, W, NV>), io::groups((a.rows + 4 / W - 1) / (4 / W)),
                           dim3(kT), 0, stream, a);
    else
        hipLaunchKernelGGL((norm_bwd_reg_kernel<Tin, Tres, Tout, W, NV>), dim3(a.blocks), dim3(kT), 0, stream, a);
    return hipGetLastError();
}

template <bool FWD, typename Tin, typename Tres, typename Tout>
hipError_t by_size(const NormArgs& a, int waves, int pieces, hipStream_t stream) {
    if (waves == 4) {
        if (pieces == 2) return reg<FWD, Tin, Tres, Tout, 4, 2>(a, stream);
        return pieces == 3 ? reg<FWD, Tin, Tres, Tout, 4, 3>(a, stream) : reg<FWD, Tin, Tres, Tout, 4, 4>(a, stream);
    }
    switch (pieces) {
        case 1: return reg<FWD, Tin, Tres, Tout, 1, 1>(a, stream);
        case 2: return reg<FWD, Tin, Tres, Tout, 1, 2>(a, stream);
        case 3: return reg<FWD, Tin, Tres, Tout, 1, 3>(a, stream);
        case 4: return reg<FWD, Tin, Tres, Tout, 1, 4>(a, stream);
        default: return reg<FWD, Tin, Tres, Tout, 1, 5>(a, stream);
    }
}

template <typename Tin, typename Tres, typename Tout>
hipError_t fwd(const NormArgs& a, hipStream_t stream) {
    int waves = 0;
    if (const int pieces = reg_pieces(a, waves)) return by_size<true, Tin, Tres, Tout>(a, waves, pieces, stream);
    KTime kt("norm_fwd", stream);
    hipLaunchKernelGGL((norm_fwd_kernel<Tin, Tres, Tout>), io::groups(a.rows), dim3(kT), 0, stream, a);
    return hipGetLastError();
}

template <typename Tin, typename Tres, typename Tout>
hipError_t bwd(const NormArgs& a, hipStream_t stream) {
    int waves = 0;
    const bool sums = a.dweight || a.dbias;
    int n = a.blocks;   // partial rows
    if (const int pieces = reg_pieces(a, waves)) {
        const hipError_t e = by_size<false, Tin, Tres, Tout>(a, waves, pieces, stream);
        if (e != hipSuccess || !sums) return e;
    } else {
        if (a.y || a.res_out) {
            KTime kt("norm_bwd", stream);
            hipLaunchKernelGGL((norm_bwd_kernel<Tin, Tres, Tout>), io::groups(a.rows), dim3(kT), 0, stream, a);
        }
        if (!sums) return hipGetLastError();
        KTime kt("norm_wgrad", stream);
        n = std::min(n, kBlocks);
        hipLaunchKernelGGL((norm_wgrad_kernel<Tres, Tout>), dim3((unsigned)((a.dim + kT - 1) / kT), n), dim3(kT), 0,
                           stream, a);
    }
    KTime kt("norm_wsum", stream);
    const unsigned columns = (unsigned)((a.dim + 63) / 64);
    const float* part = a.part;
    if (n > kSumRows) {   // (n past kBlocks: sums of kSumRows first, behind the rows)
        float* next = a.part + 2 * (int64_t)n * a.dim;
        const int slices = (n + kSumRows - 1) / kSumRows;
        hipLaunchKernelGGL(norm_wsum_kernel, dim3(columns, slices), dim3(1024), 0, stream, part, n, a.dim, next, next + a.dim);
        part = next;
        n = slices;
    }
    hipLaunchKernelGGL(norm_wsum_kernel, dim3(columns), dim3(1024), 0, stream, part, n, a.dim, a.dweight, a.dbias);
    return hipGetLastError();
}

template <bool FWD, typename Tin, typename Tres>
hipError_t by_out(const NormArgs& a, int out_bf16, hipStream_t st) {
    if constexpr (FWD) return out_bf16 ? fwd<Tin, Tres, uint16_t>(a, st) : fwd<Tin, Tres, float>(a, st);
    else return out_bf16 ? bwd<Tin, Tres, uint16_t>(a, st) : bwd<Tin, Tres, float>(a, st);
}

template <bool FWD>
hipError_t by_type(const NormArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t st) {
    if (in_bf16) return res_bf16 ? by_out<FWD, uint16_t, uint16_t>(a, out_bf16, st) : by_out<FWD, uint16_t, float>(a, out_bf16, st);
    return res_bf16 ? by_out<FWD, float, uint16_t>(a, out_bf16, st) : by_out<FWD, float, float>(a, out_bf16, st);
}

}  // namespace

// Workgroups of the gradients' kernel, each with a partial row of dweight and
// dbias: enough for the whole GPU (2 per unit for the register kernel, whose
// workgroup takes the row whole), and for the register kernel's waves to add
// up 64 rows at most; no more than have rows to work on.
int norm_bwd_blocks(int64_t rows, int64_t dim) {
    int64_t n = kBlocks;
    if (dim > 8192) n = (2048 * kT + dim - 1) / dim;
    else n = std::max(n, std::min((rows + 64 * rows_at_once(dim) - 1) / (64 * rows_at_once(dim)), (int64_t)1 << 23));
    return (int)std::min(n, (rows + rows_at_once(dim) - 1) / rows_at_once(dim));
}

size_t norm_bwd_part_bytes(int64_t rows, int64_t dim) {
    const int64_t n = norm_bwd_blocks(rows, dim);
    return (size_t)(n + (n > kSumRows ? (n + kSumRows - 1) / kSumRows : 0)) * 2 * (size_t)dim * 4;
}

hipError_t launch_norm_fwd(const NormArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t stream) {
    return by_type<true>(a, in_bf16, res_bf16, out_bf16, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t stream) {
    return by_type<false>(a, in_bf16, res_bf16, out_bf16, stream);
}

}  // namespace selscan
