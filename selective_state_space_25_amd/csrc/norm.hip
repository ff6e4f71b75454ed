// norm.hip -- layer norm with the dropout and the residual sum in front of
// it, forward and gradients.
//
//   s = dropout(x) + residual;  y = (s - mean) rstd weight + bias
//   ds = rstd (w - mean_d w - xhat mean_d (w xhat)) + dresidual,  w = dy weight
//   dweight = sum_r dy xhat;  dbias = sum_r dy
//
// One workgroup per row; the variance is summed over (s - mean)^2, not taken
// as a difference of moments.
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
    const int64_t row = blockIdx.x;
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
    const int64_t row = blockIdx.x;
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

// Partial sums of dweight and dbias: workgroup (x, y) takes 256 columns and
// every gridDim.y-th row.
template <typename Tres, typename Tout>
__global__ __launch_bounds__(kT) void norm_wgrad_kernel(NormArgs a) {
    const int64_t d = (int64_t)blockIdx.x * kT + threadIdx.x;
    if (d >= a.dim) return;
    const Tout* DY = reinterpret_cast<const Tout*>(a.x) + d;
    const Tres* S = reinterpret_cast<const Tres*>(a.res) + d;
    float gw = 0.0f, gb = 0.0f;
    for (int64_t r = blockIdx.y; r < a.rows; r += a.blocks) {
        const float dy = io::ld(DY + r * a.dim);
        gw += dy * ((io::ld(S + r * a.dim) - a.mean_in[r]) * a.rstd_in[r]);
        gb += dy;
    }
    a.part[(2 * (int64_t)blockIdx.y) * a.dim + d] = gw;
    a.part[(2 * (int64_t)blockIdx.y + 1) * a.dim + d] = gb;
}

__global__ __launch_bounds__(kT) void norm_wsum_kernel(NormArgs a) {
    const int64_t d = (int64_t)blockIdx.x * kT + threadIdx.x;
    if (d >= a.dim) return;
    float gw = 0.0f, gb = 0.0f;
    for (int b = 0; b < a.blocks; ++b) {
        gw += a.part[(2 * (int64_t)b) * a.dim + d];
        gb += a.part[(2 * (int64_t)b + 1) * a.dim + d];
    }
    if (a.dweight) a.dweight[d] = gw;
    if (a.dbias) a.dbias[d] = gb;
}

template <typename Tin, typename Tres, typename Tout>
hipError_t fwd(const NormArgs& a, hipStream_t stream) {
    KTime kt("norm_fwd", stream);
    hipLaunchKernelGGL((norm_fwd_kernel<Tin, Tres, Tout>), dim3((unsigned)a.rows), dim3(kT), 0, stream, a);
    return hipGetLastError();
}

template <typename Tin, typename Tres, typename Tout>
hipError_t bwd(const NormArgs& a, hipStream_t stream) {
    if (a.y || a.res_out) {
        KTime kt("norm_bwd", stream);
        hipLaunchKernelGGL((norm_bwd_kernel<Tin, Tres, Tout>), dim3((unsigned)a.rows), dim3(kT), 0, stream, a);
    }
    if (a.dweight || a.dbias) {
        const unsigned cols = (unsigned)((a.dim + kT - 1) / kT);
        {
            KTime kt("norm_wgrad", stream);
            hipLaunchKernelGGL((norm_wgrad_kernel<Tres, Tout>), dim3(cols, a.blocks), dim3(kT), 0, stream, a);
        }
        KTime kt("norm_wsum", stream);
        hipLaunchKernelGGL(norm_wsum_kernel, dim3(cols), dim3(kT), 0, stream, a);
    }
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

// Row slices that the weight gradients are summed in.
int norm_bwd_blocks(int64_t rows, int64_t dim) {
    const int64_t cols = (dim + kT - 1) / kT;
    int64_t n = (2048 + cols - 1) / cols;
    if (n > rows) n = rows;
    return (int)n;
}

hipError_t launch_norm_fwd(const NormArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t stream) {
    return by_type<true>(a, in_bf16, res_bf16, out_bf16, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t stream) {
    return by_type<false>(a, in_bf16, res_bf16, out_bf16, stream);
}

}  // namespace selscan
