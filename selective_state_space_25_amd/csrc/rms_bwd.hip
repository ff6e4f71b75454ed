// rms_bwd.hip -- gradients of the RMS norm, for gfx950.
//
//   w = dy weight;  xhat = s rstd
//   ds = rstd (w - xhat sum (w xhat) / width) + dresidual
//   without a gate: dx = ds, dresidual = ds
//   with one: dx = ds silu(z), dz = ds x silu'(z)      (s = x silu(z) made again)
//   dweight = sum over rows of dy xhat
//
// A stream bound by memory, laid out as the forward is (rms_rows.hpp): a group
// stays in registers between its sum and its gradients.  A workgroup walks the
// rows of one group of columns a fixed distance apart and keeps its sums for
// dweight in registers, 64 rows in fp32 at most (there are more workgroups
// where there are more rows), one partial row a workgroup, which
// column_sums.hip adds in fp64: a fixed order.
//
// 32768 x 2560, bf16 with an fp32 residual: 249 us for 1.34 GB, 5.4 TB/s, and
// 5 us for the partial rows.  With a gate 225 us there and 211 at 16384 x 5120
// for 0.84 GB, 3.7 and 4.0 TB/s: waves wait half their time and more for loads,
// with fewer of them on a compute unit (registers).
#include <algorithm>

#include "rms_rows.hpp"

namespace selscan {

namespace {

using namespace rms;

constexpr int kBlocks = 512;

// Groups of up to 2560 elements stay in one wave: three or four streams of
// loads a group are enough without a barrier.  us, one wave / four, 84
// million elements in bf16:
//                          1280         2048         2560
//   with fp32 residual   265 / 272    251 / 282    253 / 336
//   with a gate          210 / 252    253 / 248    230 / 292
// Longer ones take four: 333 and 301 just past it (2568, a third of the lanes
// idle), 254 and 221 at 4096, 246 and 268 at 8192.
constexpr int kWavePieces = 320;

// One group of one row.  GATE: res is x, in Tin.
template <typename Tin, typename Tres, typename Tout, bool GATE>
struct Row {
    const Tout* dy;
    const Tres* s;
    const Tin* z;
    const float* w;
    const Tres* dr;
    Tin *dx, *dz;
    Tres* ds;
    float rstd;
    int width;
    __device__ __forceinline__ Row(const RmsArgs& a, int64_t row, int64_t g) {
        const int64_t base = row * a.dim + g * a.width;
        dy = static_cast<const Tout*>(a.x) + base;
        s = static_cast<const Tres*>(a.res) + base;
        z = GATE ? static_cast<const Tin*>(a.gate) + row * a.gate_row + g * a.width : nullptr;
        w = a.weight ? a.weight + g * a.width : nullptr;
        dr = a.dres_in ? static_cast<const Tres*>(a.dres_in) + base : nullptr;
        dx = a.y ? static_cast<Tin*>(a.y) + base : nullptr;
        dz = a.dgate ? static_cast<Tin*>(a.dgate) + base : nullptr;
        ds = a.res_out ? static_cast<Tres*>(a.res_out) + base : nullptr;
        rstd = a.rstd_in[row * a.groups + g];
        width = (int)a.width;
    }
    // dy, x (or s) and z of the piece from element d
    template <bool FULL>
    __device__ __forceinline__ void load(int d, float (&y)[8], float (&x)[8], float (&zv)[GATE ? 8 : 1]) const {
        ldp<FULL>(dy + d, width - d, y);
        ldp<FULL>(s + d, width - d, x);
        if constexpr (GATE) ldp<FULL>(z + d, width - d, zv);
    }
    __device__ __forceinline__ float xhat(float x, float zv) const {
        if constexpr (GATE) x *= silu_scaled(zv, 1.0f);
        return x * rstd;
    }
    // from y = dy: the piece's share of the sum, and of dweight
    template <bool FULL>
    __device__ __forceinline__ float dot(int d, float (&y)[8], const float (&x)[8], const float (&zv)[GATE ? 8 : 1],
                                         float* gw) const {
        float t[8], c = 0.0f;
        if (w) ldp<FULL>(w + d, width - d, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xh = xhat(x[i], zv[GATE ? i : 0]);
            if (gw) gw[i] = __builtin_fmaf(y[i], xh, gw[i]);
            if (w) y[i] *= t[i];
            c = __builtin_fmaf(y[i], xh, c);
        }
        return c;
    }
    // the gradients, from y = w and c = the sum over the group / width
    template <bool FULL>
    __device__ __forceinline__ void store(int d, float c, float (&y)[8], const float (&x)[8], const float (&zv)[GATE ? 8 : 1]) const {
        float t[8];
        if (dr) ldp<FULL>(dr + d, width - d, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = (y[i] - xhat(x[i], zv[GATE ? i : 0]) * c) * rstd;
            if (dr) y[i] += t[i];
        }
        if constexpr (GATE) {
            float g[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float sg = sigmoid(zv[i]);
                g[i] = y[i] * x[i] * (sg * __builtin_fmaf(zv[i], 1.0f - sg, 1.0f));
                y[i] *= zv[i] * sg;
            }
            if (dz) stp<FULL>(dz + d, width - d, g);
        } else {
            if (ds) stp<FULL>(ds + d, width - d, y);
        }
        if (dx) stp<FULL>(dx + d, width - d, y);
    }
};

template <typename Tin, typename Tres, typename Tout, bool GATE, int LR, int NV>
__global__ __launch_bounds__(kT) void rms_bwd_kernel(RmsArgs a) {
    __shared__ float sm[4];
    __shared__ __attribute__((aligned(16))) float sums[LR < 256 ? kT * 8 : 1];
    constexpr int kRows = kT / LR;
    const int at = threadIdx.x % LR;
    const int64_t g = blockIdx.y;
    const bool outs = a.y || a.res_out || a.dgate;
    float gw[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) gw[j][i] = 0.0f;
    for (int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / LR; r < a.rows; r += (int64_t)gridDim.x * kRows) {
        const Row<Tin, Tres, Tout, GATE> row(a, r, g);
        float y[NV][8], x[NV][8], z[NV][GATE ? 8 : 1];
        float c = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = 8 * (at + LR * j);
            if (j + 1 < NV) row.template load<true>(d, y[j], x[j], z[j]);
            else if (d < row.width) row.template load<false>(d, y[j], x[j], z[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = 8 * (at + LR * j);
            if (j + 1 < NV) c += row.template dot<true>(d, y[j], x[j], z[j], gw[j]);
            else if (d < row.width) c += row.template dot<false>(d, y[j], x[j], z[j], gw[j]);
        }
        if (!outs) continue;
        c = row_sum<LR>(c, sm) * a.inv_width;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = 8 * (at + LR * j);
            if (j + 1 < NV) row.template store<true>(d, c, y[j], x[j], z[j]);
            else if (d < row.width) row.template store<false>(d, c, y[j], x[j], z[j]);
        }
    }
    if (!a.part) return;
    float* out = a.part + (int64_t)blockIdx.x * a.dim + g * a.width;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int d = 8 * (at + LR * j);
        if constexpr (LR == 256) {
            if (d < a.width) stp<false>(out + d, (int)a.width - d, gw[j]);
        } else {   // the workgroup's rows' sums of the same columns, in their order
            __syncthreads();
            io::st8(sums + threadIdx.x * 8, gw[j]);
            __syncthreads();
            for (int e = threadIdx.x; e < LR * 8 && LR * 8 * j + e < a.width; e += kT) {
                float v = sums[e];
                for (int i = 1; i < kRows; ++i) v += sums[i * LR * 8 + e];
                out[LR * 8 * j + e] = v;
            }
        }
    }
}

// Groups longer than the registers: read twice (sums as in the forward), and
// dweight by columns.
template <typename Tin, typename Tres, typename Tout, bool GATE>
__global__ __launch_bounds__(kT) void rms_bwd_long_kernel(RmsArgs a) {
    __shared__ float sm[4];
    const int64_t unit = io::group_id(), r = unit / a.groups;
    if (r >= a.rows) return;
    const Row<Tin, Tres, Tout, GATE> row(a, r, unit - r * a.groups);
    float y[8], x[8], z[GATE ? 8 : 1];
    double sum = 0.0;
    for (int d = 8 * (int)threadIdx.x; d < row.width; d += 8 * kT) {
        row.template load<false>(d, y, x, z);
        sum += row.template dot<false>(d, y, x, z, nullptr);
    }
    const float c = row_sum<256>((float)sum, sm) * a.inv_width;
    for (int d = 8 * (int)threadIdx.x; d < row.width; d += 8 * kT) {
        row.template load<false>(d, y, x, z);
        row.template dot<false>(d, y, x, z, nullptr);
        row.template store<false>(d, c, y, x, z);
    }
}

// Workgroup (x, y, g): 2048 columns of group g, every gridDim.y-th row.
template <typename Tin, typename Tres, typename Tout, bool GATE>
__global__ __launch_bounds__(kT) void rms_wgrad_kernel(RmsArgs a) {
    const int d = 8 * (int)(blockIdx.x * kT + threadIdx.x);
    const int64_t g = blockIdx.z;
    if (d >= a.width) return;
    float gw[8] = {};
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const Row<Tin, Tres, Tout, GATE> row(a, r, g);
        float y[8], x[8], z[GATE ? 8 : 1];
        row.template load<false>(d, y, x, z);
        row.template dot<false>(d, y, x, z, gw);
    }
    stp<false>(a.part + (int64_t)blockIdx.y * a.dim + g * a.width + d, (int)a.width - d, gw);
}

template <typename Tin, typename Tres, typename Tout, bool GATE>
struct Bwd {
    const RmsArgs& a;
    hipStream_t stream;
    template <int LR, int NV>
    hipError_t run() {
        KTime kt("rms_bwd", stream);
        hipLaunchKernelGGL((rms_bwd_kernel<Tin, Tres, Tout, GATE, LR, NV>), dim3(a.blocks, (unsigned)a.groups), dim3(kT), 0,
                           stream, a);
        return hipGetLastError();
    }
};

template <typename Tin, typename Tres, typename Tout, bool GATE>
hipError_t bwd(const RmsArgs& a, hipStream_t stream) {
    const Layout l(a.width, kWavePieces);
    if (l.pieces) return by_layout<5, 5>(l, Bwd<Tin, Tres, Tout, GATE>{a, stream});
    if (a.y || a.res_out || a.dgate) {
        KTime kt("rms_bwd", stream);
        hipLaunchKernelGGL((rms_bwd_long_kernel<Tin, Tres, Tout, GATE>), io::groups(a.rows * a.groups), dim3(kT), 0, stream, a);
    }
    if (a.part) {
        KTime kt("rms_wgrad", stream);
        hipLaunchKernelGGL((rms_wgrad_kernel<Tin, Tres, Tout, GATE>),
                           dim3((unsigned)((a.width + 8 * kT - 1) / (8 * kT)), a.blocks, (unsigned)a.groups), dim3(kT), 0, stream, a);
    }
    return hipGetLastError();
}

template <typename Tin, typename Tres>
hipError_t by_out(const RmsArgs& a, int out_bf16, hipStream_t st) {
    if constexpr (sizeof(Tin) == sizeof(Tres)) {
        if (a.gate) return out_bf16 ? bwd<Tin, Tin, uint16_t, true>(a, st) : bwd<Tin, Tin, float, true>(a, st);
    }
    return out_bf16 ? bwd<Tin, Tres, uint16_t, false>(a, st) : bwd<Tin, Tres, float, false>(a, st);
}

}  // namespace

// Workgroups to a group of columns, each with a partial row of dweight: two a
// compute unit, and 64 rows each in fp32 at most; no more than have rows.
int rms_bwd_blocks(int64_t rows, int64_t width) {
    const Layout l(width, kWavePieces);
    const int64_t once = l.at_once();
    const int64_t n = l.pieces ? std::max((int64_t)kBlocks, std::min((rows + 64 * once - 1) / (64 * once), (int64_t)1 << 23))
                               : std::max((int64_t)64, std::min((rows + 63) / 64, (int64_t)65535));
    return (int)std::min(n, (rows + once - 1) / once);
}

bool rms_reads_again(int64_t width) { return !Layout(width, kWavePieces).pieces; }

size_t rms_bwd_part_bytes(int64_t rows, int64_t dim, int64_t groups) {
    return (size_t)column_sums_rows(rms_bwd_blocks(rows, dim / groups)) * (size_t)dim * 4;
}

hipError_t launch_rms_bwd(const RmsArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t stream) {
    hipError_t e;
    if (in_bf16) e = res_bf16 ? by_out<uint16_t, uint16_t>(a, out_bf16, stream) : by_out<uint16_t, float>(a, out_bf16, stream);
    else e = res_bf16 ? by_out<float, uint16_t>(a, out_bf16, stream) : by_out<float, float>(a, out_bf16, stream);
    if (e != hipSuccess || !a.part) return e;
    KTime kt("rms_wsum", stream);
    return launch_column_sums(a.part, a.blocks, a.dim, 0, a.dweight, nullptr, stream);
}

}  // namespace selscan
