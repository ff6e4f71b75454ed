// short_conv.hip -- short causal convolution of token-major rows, its
// gradients and its one-token form, for gfx950.
//
//   pre_t = bias + sum_k w[k] x_{t-K+1+k};   out_t = act(pre_t),   act = silu or identity
//   g_t   = dout_t act'(pre_t);   dx_s = sum_k w[k] g_{s+K-1-k}
//   dw[k] = sum_t g_t x_{t-K+1+k};   dbias = sum_t g_t
//
// per channel, K taps (2, 3 or 4), the K - 1 tokens before the first from a
// state.  Streams bound by memory: x in and out out; x, dout in and dx out.  A
// thread owns V neighbouring channels and walks a run of tokens with the last
// K - 1 inputs (and gradients g) in registers, so an element is read once but
// for the K - 1 tokens at a run's edges.  A workgroup is a power of two of such
// columns by as many runs as make 256 threads: with columns narrower than a
// wave, few channels still fill it.  Rows may start at any element's address
// (16-byte accesses are allowed there), which a slice of a projection's result
// does.  The gradients' recompute pre from x.  dw and dbias: fp32 over one
// run, the workgroup's runs added up through LDS, one partial row a workgroup,
// and those in fp64 by column_sums.hip in a fixed order.
//
// 8 x 4096 x 2304, width 4, split in three, bf16: 61 us for 0.30 GB, 5.0 TB/s
// (fp32 123 for 0.60); gradients with dout in fp32 137 us for 0.60 GB, 4.4 TB/s
// (vector ALU 73 % busy: the activation and its slope again, 2 K multiplications
// an element; x in fp32 183 for 0.91).  One token is a launch: 2.1 us at 1 x
// 2304, 5.1 at 128 x 2304.
#include "io.hpp"
#include "kernels.hpp"

namespace selscan {

namespace {

constexpr int kT = 256;
constexpr int kFwdU = 4, kBwdU = 4;   // tokens asked for at a time

// A thread's place: V channels from c of batch element b, tokens t0 .. t1 - 1.
struct Place {
    int64_t b, c, t0, t1, len;
    bool live;
    int col, run;       // column and run inside the workgroup
    int64_t block;      // (batch, token block): the partial row of the gradients
    __device__ __forceinline__ Place(const ShortConvArgs& a, int V) {
        const int64_t g = io::group_id();
        const int64_t cb = g % a.col_blocks;
        block = g / a.col_blocks;
        b = block / a.run_blocks;
        col = (int)(threadIdx.x & (a.cols - 1));
        run = (int)(threadIdx.x / a.cols);
        c = (cb * a.cols + col) * V;
        const int64_t runs = kT / a.cols;
        t0 = ((block - b * a.run_blocks) * runs + run) * a.run;
        t1 = min(t0 + a.run, a.L);
        live = b < a.batch && c < a.C && t0 < a.L;
        len = a.L;
        if (a.lengths && b < a.batch) len = min((int64_t)max(a.lengths[b], 0), a.L);
    }
};

// The taps of V channels.
template <int K, int V>
__device__ __forceinline__ void taps(const ShortConvArgs& a, int64_t c, float (&w)[K][V], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = a.bias ? a.bias[c + i] : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][i] = a.weight[(c + i) * K + k];
    }
}

// Input token t >= -(K - 1), from the state where it is negative.
template <typename Tin, int K, int V>
__device__ __forceinline__ void input(const ShortConvArgs& a, const Place& p, const Tin* X, int64_t t, io::Piece<Tin, V>& r) {
    if (t >= 0) {
        if (t < p.len) r.get(X + t * a.x_row);
        else r.zero();
    } else if (a.state) {
        r.get(static_cast<const Tin*>(a.state) + (p.b * (K - 1) + t + K - 1) * a.C + p.c);
    } else {
        r.zero();
    }
}

// The piece of the split rows (y or dout) that the V channels from c lie in:
// its address at batch element b's first token, and its row.
template <typename T>
__device__ __forceinline__ T* part_of(const ShortConvArgs& a, T* p0, T* p1, T* p2, int64_t b, int64_t c, int64_t& row) {
    const int i = c < a.begin[1] ? 0 : c < a.begin[2] ? 1 : 2;
    row = i == 0 ? a.begin[1] : i == 1 ? a.begin[2] - a.begin[1] : a.C - a.begin[2];
    T* p = i == 0 ? p0 : i == 1 ? p1 : p2;
    return p + b * a.L * row + (c - (i == 0 ? 0 : i == 1 ? a.begin[1] : a.begin[2]));
}

template <typename Tin, typename Tout, int K, int V>
__global__ __launch_bounds__(kT) void conv_fwd_kernel(ShortConvArgs a) {
    constexpr int kU = kFwdU;
    const Place p(a, V);
    if (!p.live) return;
    const Tin* X = static_cast<const Tin*>(a.x) + p.b * a.x_batch + p.c;
    int64_t row;
    Tout* Y = part_of(a, static_cast<Tout*>(a.y[0]), static_cast<Tout*>(a.y[1]), static_cast<Tout*>(a.y[2]), p.b, p.c, row);
    float w[K][V], bias[V];
    taps(a, p.c, w, bias);
    float xs[K - 1 + kU][V];
    io::Piece<Tin, V> next[kU];
    const int64_t te = min(p.t1, p.len);
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (t + u < te) next[u].get(X + (t + u) * a.x_row);
    };
#pragma unroll
    for (int u = 0; u < kU; ++u) next[u].zero();
    fetch(p.t0);
    if (p.t0 < te) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            io::Piece<Tin, V> r;
            input<Tin, K, V>(a, p, X, p.t0 - (K - 1) + j, r);
            r.widen(xs[j]);
        }
    }
    for (int64_t t = p.t0; t < te; t += kU) {
#pragma unroll
        for (int u = 0; u < kU; ++u) next[u].widen(xs[K - 1 + u]);
        fetch(t + kU);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (t + u >= te) break;
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float pre = bias[i];
#pragma unroll
                for (int k = 0; k < K; ++k) pre = __builtin_fmaf(w[k][i], xs[u + k][i], pre);
                y[i] = a.silu ? silu_scaled(pre, 1.0f) : pre;
            }
            io::Piece<Tout, V> o;
            o.narrow(y);
            o.put(Y + (t + u) * row);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) xs[j][i] = xs[kU + j][i];
    }
    io::Piece<Tout, V> none;
    none.zero();
    for (int64_t t = max(p.t0, p.len); t < p.t1; ++t) none.put(Y + t * row);
    if (p.t0 == 0 && a.last) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            io::Piece<Tin, V> r;
            input<Tin, K, V>(a, p, X, p.len - (K - 1) + j, r);
            r.put(static_cast<Tin*>(a.last) + (p.b * (K - 1) + j) * a.C + p.c);
        }
    }
}

template <typename Tin, typename Tout, int K, int V>
__global__ __launch_bounds__(kT) void conv_bwd_kernel(ShortConvArgs a) {
    constexpr int kU = kBwdU;
    __shared__ float sums[(K + 1) * V][kT];
    const Place p(a, V);
    float dw[K + 1][V];   // of the taps, then of the bias
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[k][i] = 0.0f;
    if (p.live) {
        const Tin* X = static_cast<const Tin*>(a.x) + p.b * a.x_batch + p.c;
        Tin* DX = static_cast<Tin*>(a.dx) + p.b * a.L * a.C + p.c;
        const int64_t srow = p.b * (K - 1) * a.C + p.c;
        int64_t row;
        const Tout* DY = part_of(a, static_cast<const Tout*>(a.dout[0]), static_cast<const Tout*>(a.dout[1]),
                                 static_cast<const Tout*>(a.dout[2]), p.b, p.c, row);
        float w[K][V], bias[V];
        taps(a, p.c, w, bias);
        float xs[K - 1 + kU][V], gs[K - 1 + kU][V];
        io::Piece<Tin, V> nx[kU];
        io::Piece<Tout, V> ny[kU];
        // g reaches K - 1 tokens past the run
        const int64_t tg = min(p.t1 + K - 1, p.len), tw = min(p.t1, p.len);
        auto fetch = [&](int64_t t) {
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (t + u < tg) {
                    nx[u].get(X + (t + u) * a.x_row);
                    ny[u].get(DY + (t + u) * row);
                }
        };
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            nx[u].zero();
            ny[u].zero();
        }
        fetch(p.t0);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            io::Piece<Tin, V> r;
            input<Tin, K, V>(a, p, X, p.t0 - (K - 1) + j, r);
            r.widen(xs[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) gs[j][i] = 0.0f;
        }
        // a run's own g before t0 belongs to the runs before: dx starts at t0,
        // whose sum needs no earlier g; the first run goes on to the state's
        for (int64_t t = p.t0; t < p.t1 + K - 1; t += kU) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                nx[u].widen(xs[K - 1 + u]);
                ny[u].widen(gs[K - 1 + u]);
            }
            fetch(t + kU);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (t + u >= p.t1 + K - 1) break;
                float (&g)[V] = gs[K - 1 + u];
                if (t + u < tg) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float pre = bias[i];
#pragma unroll
                        for (int k = 0; k < K; ++k) pre = __builtin_fmaf(w[k][i], xs[u + k][i], pre);
                        const float s = fast_rcp(1.0f + fast_exp2(-pre * kLog2e));
                        if (a.silu) g[i] *= s * __builtin_fmaf(pre, 1.0f - s, 1.0f);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) g[i] = 0.0f;
                }
                if (t + u < tw) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][i] = __builtin_fmaf(g[i], xs[u + k][i], dw[k][i]);
                        dw[K][i] += g[i];
                    }
                }
                const int64_t s = t + u - (K - 1);
                if (s < p.t0 && (s >= 0 || !a.dstate)) continue;
                float d[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    d[i] = 0.0f;
#pragma unroll
                    for (int k = 0; k < K; ++k) d[i] = __builtin_fmaf(w[k][i], gs[K - 1 + u - k][i], d[i]);
                }
                if (a.dlast && s < p.len && s >= p.len - (K - 1)) {
                    io::Piece<Tin, V> r;
                    float e[V];
                    r.get(static_cast<const Tin*>(a.dlast) + srow + (s - (p.len - (K - 1))) * a.C);
                    r.widen(e);
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] += e[i];
                }
                io::Piece<Tin, V> o;
                o.narrow(d);
                if (s >= p.len) o.zero();   // (past the end)
                o.put(s >= 0 ? DX + s * a.C : static_cast<Tin*>(a.dstate) + srow + (s + K - 1) * a.C);
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xs[j][i] = xs[kU + j][i];
                    gs[j][i] = gs[kU + j][i];
                }
        }
    }
    if (!a.part) return;
    // the runs' sums of the same column, in their order
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sums[k * V + i][threadIdx.x] = dw[k][i];
    __syncthreads();
    if (p.b >= a.batch) return;
    const int64_t c0 = p.c - (int64_t)p.col * V;
    float* out = a.part + p.block * (K + 1) * a.C;
    for (int e = threadIdx.x; e < (K + 1) * V * a.cols; e += kT) {
        // [channels, K], then [channels]
        const bool tap = e < K * V * a.cols;
        const int ci = tap ? e / K : e - K * V * a.cols, k = tap ? e - ci * K : K;
        float v = 0.0f;
        for (int r = 0; r < kT / a.cols; ++r) v += sums[k * V + ci % V][r * a.cols + ci / V];
        const int64_t c = c0 + ci;
        if (c < a.C) out[tap ? c * K + k : K * a.C + c] = v;
    }
}

// One token: x [batch, C], the state moved on in place by the threads that own its channels.
template <typename Tin, typename Tout, int K, int V>
__global__ __launch_bounds__(kT) void conv_step_kernel(ShortConvArgs a) {
    const int64_t id = io::group_id() * kT + threadIdx.x, n = a.C / V;
    const int64_t b = id / n, c = (id - b * n) * V;
    if (b >= a.batch) return;
    Tin* S = static_cast<Tin*>(a.last) + b * (K - 1) * a.C + c;
    io::Piece<Tin, V> r[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j].get(S + j * a.C);
    r[K - 1].get(static_cast<const Tin*>(a.x) + b * a.x_batch + c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j + 1].put(S + j * a.C);
    if (!a.y[0]) return;   // (the state alone)
    float w[K][V], y[V];
    taps(a, c, w, y);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float x[V];
        r[k].widen(x);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = __builtin_fmaf(w[k][i], x[i], y[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = a.silu ? silu_scaled(y[i], 1.0f) : y[i];
    io::Piece<Tout, V> o;
    o.narrow(y);
    o.put(static_cast<Tout*>(a.y[0]) + b * a.C + c);
}

enum Form { kFwd, kBwd, kStep };

template <Form F, typename Tin, typename Tout, int K, int V>
hipError_t launch_v(const ShortConvArgs& a, hipStream_t stream) {
    if constexpr (F == kStep) {
        KTime kt("short_conv_step", stream);
        const int64_t threads = a.batch * (a.C / V);
        hipLaunchKernelGGL((conv_step_kernel<Tin, Tout, K, V>), io::groups((threads + kT - 1) / kT), dim3(kT), 0, stream, a);
    } else {
        const dim3 grid = io::groups(a.col_blocks * a.run_blocks * a.batch);
        KTime kt(F == kFwd ? "short_conv_fwd" : "short_conv_bwd", stream);
        if constexpr (F == kFwd) hipLaunchKernelGGL((conv_fwd_kernel<Tin, Tout, K, V>), grid, dim3(kT), 0, stream, a);
        else hipLaunchKernelGGL((conv_bwd_kernel<Tin, Tout, K, V>), grid, dim3(kT), 0, stream, a);
    }
    return hipGetLastError();
}

// Channels a thread has at a time: whole pieces of the split only, one where
// those are not (2303 channels in bf16: 96 us where 2304 take 60, gradients 185
// and 139).  Twice as many take 73 us at the sizes above (fewer waves to hide
// loads behind), and 150 for the gradients.
constexpr int kFwdV = 4, kBwdV = 2;

template <Form F, typename Tin, typename Tout, int K>
hipError_t by_v(const ShortConvArgs& a, hipStream_t stream) {
    constexpr int V = F == kBwd ? kBwdV : kFwdV;
    return a.V == V ? launch_v<F, Tin, Tout, K, V>(a, stream) : launch_v<F, Tin, Tout, K, 1>(a, stream);
}

template <Form F, typename Tin, typename Tout>
hipError_t by_k(const ShortConvArgs& a, hipStream_t stream) {
    return a.K == 2 ? by_v<F, Tin, Tout, 2>(a, stream) : a.K == 3 ? by_v<F, Tin, Tout, 3>(a, stream) : by_v<F, Tin, Tout, 4>(a, stream);
}

template <Form F>
hipError_t by_type(const ShortConvArgs& a, int in_bf16, int out_bf16, hipStream_t st) {
    if (in_bf16) return out_bf16 ? by_k<F, uint16_t, uint16_t>(a, st) : by_k<F, uint16_t, float>(a, st);
    return out_bf16 ? by_k<F, float, uint16_t>(a, st) : by_k<F, float, float>(a, st);
}

}  // namespace

// How the threads divide the work: V channels each, `cols` columns and
// kT / cols runs of `run` tokens a workgroup.
void short_conv_plan(ShortConvArgs& a, bool bwd) {
    const int V = bwd ? kBwdV : kFwdV;
    const bool whole = a.begin[1] % V == 0 && a.begin[2] % V == 0 && a.C % V == 0;
    a.V = whole ? V : 1;
    const int64_t n = a.C / a.V;
    // the fewest idle columns; of as many, the widest
    a.cols = 64;
    for (int c = 32; c >= 8; c /= 2)
        if ((n + c - 1) / c * c < (n + a.cols - 1) / a.cols * a.cols) a.cols = c;
    a.col_blocks = (n + a.cols - 1) / a.cols;
    // long runs read fewer tokens twice; shorter ones where the GPU would not fill
    // (a wave to each SIMD is 2^16 threads; loads need a few waves)
    a.run = 32;
    while (a.run > 4 && a.batch * ((a.L + a.run - 1) / a.run) * a.col_blocks * a.cols < (int64_t)1 << 18) a.run /= 2;
    const int64_t runs = (a.L + a.run - 1) / a.run;
    a.run_blocks = (runs + kT / a.cols - 1) / (kT / a.cols);
}

hipError_t launch_short_conv_fwd(const ShortConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream) {
    return by_type<kFwd>(a, in_bf16, out_bf16, stream);
}
hipError_t launch_short_conv_bwd(const ShortConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream) {
    const hipError_t e = by_type<kBwd>(a, in_bf16, out_bf16, stream);
    if (e != hipSuccess || !a.part) return e;
    KTime kt("short_conv_wsum", stream);
    return launch_column_sums(a.part, a.batch * a.run_blocks, a.K * a.C, a.C, a.dweight, a.dbias, stream);
}
hipError_t launch_short_conv_step(const ShortConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream) {
    return by_type<kStep>(a, in_bf16, out_bf16, stream);
}

}  // namespace selscan
