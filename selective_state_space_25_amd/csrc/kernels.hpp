// kernels.hpp -- argument blocks and launchers shared by the host entry
// points and the HIP kernels (internal to libselscan; not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "selscan.h"

namespace selscan {

// Records `msg` as the calling thread's selscan_last_error() and returns s.
selscan_status_t set_error(selscan_status_t s, const std::string& msg);

// Per-kernel timing bracket (no-op unless selscan_timing_enable(1)).
void ktime_mark(const char* kernel, hipStream_t stream, bool begin);
struct KTime {
    const char* name;
    hipStream_t stream;
    KTime(const char* n, hipStream_t s) : name(n), stream(s) { ktime_mark(name, stream, true); }
    ~KTime() { ktime_mark(name, stream, false); }
};

// Mamba-1.  Tensors as in selscan.h; ws_* point into the workspace.
struct M1Args {
    const void* u;
    const void* delta;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* z;
    const float* bias;
    void* y;
    float* last;
    const float* h0;  // [batch, dim, N] initial state, or NULL for zero
    float* ws_state;  // [rows, G, 16] chunk end states from a zero start
    float* ws_w;      // [rows, G] chunk sums of Delta / ln2
    float* bcq;       // [batch, L, 32] fp32 copy of B and C (B0..B15, C0..C15 per token)
    int64_t batch, dim, L;
    int64_t chunk;    // longest chunk in tokens; the kernels split a row's tiles evenly over G chunks
    int N;            // d_state
    int G;            // chunks per row
    int softplus;
    int vec_ok;       // rows of u, delta, z, y start on 16-byte boundaries (tile path)
    int force_general;
    int xcd_chunks;   // G is a multiple of 8 and chunk g runs on XCD g % 8 (1-D grid)
    int carry_scan;   // the carries come from a scan over the chunk summaries (its own
                      // kernel) rather than from a fold at the start of each chunk
};

int m1_padded_states(int N);
int m1_chunk_align(int in_bf16);
int m1_resident_waves_per_cu(int in_bf16);
int m1_rows_per_block();
int m1_waves_per_block();
size_t m1_bc_bytes(int64_t batch, int64_t L);
hipError_t launch_m1(const M1Args& a, int in_bf16, int out_bf16, hipStream_t stream);
// B, C [batch, N, L] -> bcq [batch, L, 32] fp32 records (zeros past N).
hipError_t launch_m1_bc(const void* B, const void* C, int64_t batch, int N, int64_t L, float* bcq, int in_bf16,
                        hipStream_t stream);

// Mamba-1 backward.  Inputs as for M1Args plus dout [batch, dim, L]
// (out dtype); gradients fp32 in the layouts of their inputs.  hbuf .. part
// point into the workspace (m1_bwd_carve).
struct BwdArgs {
    const void* u;
    const void* delta;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* z;
    const float* bias;
    const float* h0;
    const void* dout;
    float *du, *ddelta, *dA, *dB, *dC, *dD, *dz, *dbias, *dh0;
    float* hbuf;    // [rows, G, 16] chunk-end states from zero, then states entering each chunk
    float* mubuf;   // [rows, G, 16] adjoint leaving each chunk from zero, then the one entering it
    float* wbuf;    // [rows, G] chunk sums of Delta
    float* pA;      // [rows, G, 16] per-chunk dA terms
    float* pD;      // [rows, G]
    float* pbias;   // [rows, G]
    float* part;    // [dim / 64, batch, L, 32] per-channel-block dB (16) and dC (16)
    float* ckz;     // [batch, tiles, dim, 16] state entering every tile (m1_bwd_tile() tokens) from the chunk's zero start
    float* wck;     // [batch, tiles, dim] sum of Delta from the chunk's start to the same tokens
    float* bcq;     // [batch, L, 32] fp32 records of B and C (the lane-per-channel summary pass)
    int lane_sum;   // the summary pass runs one channel per lane (rows 16-byte aligned)
    int chunk_img;  // the chunk pass reads 32-token row images (lane_sum, bf16 inputs, L and chunk multiples of 32)
    int64_t batch, dim, L;
    int64_t chunk;  // tokens per chunk: a multiple of m1_bwd_tile(), at most m1_bwd_max_chunk()
    int64_t G;      // chunks
    int N;
    int softplus;
};
int m1_bwd_tile();
int m1_bwd_max_chunk();
int m1_bwd_channels_per_block();
size_t m1_bwd_workspace_bytes(int64_t batch, int64_t dim, int64_t L, int64_t G);
void m1_bwd_carve(BwdArgs& a, void* ws);
hipError_t launch_m1_bwd(const BwdArgs& a, int in_bf16, int out_bf16, hipStream_t stream);

// Mamba-2.
struct M2Args {
    const void* x;
    const void* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* z;
    const float* dt_bias;
    void* y;
    float* last;
    const float* h0;  // [batch, H, P, N] initial state, or NULL for zero
    float* ws_bc;     // [batch, L, G, 2, N] fp32 copy of B and C (interleaved per token)
    float* ws_state;  // [batch, H, P, chunks, N] chunk end states, then carries-in
    float* ws_w;      // [batch, H, chunks] chunk sums of Delta / ln2
    int64_t batch, L, H, P, G, N;
    int64_t chunk;
    int chunks;
    int softplus;
    int xcd_units;    // chunked matrix form: place the units of one batch on one XCD
};

int m2_waves_per_block(int64_t N);

// Mamba-2 gradients (recurrent form, headdim 64).  Tensors as in selscan.h;
// ck, pB, pC, pA, pD, pbias point into the workspace (m2_bwd_carve).
struct M2BwdArgs {
    const void* x;
    const void* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* z;
    const float* dt_bias;
    const float* h0;
    const void* dout;
    float *dx, *ddt, *dA, *dB, *dC, *dD, *dz, *ddt_bias, *dh0;
    float* ck;        // [batch*H, tiles, N/16, 4, 64, 4] states entering each 8-token tile
                      // (the chunked form: each 32-token chunk, as
                      // [batch*H, chunks, N/16, 4, 4, 16, 4]: n block, p block,
                      // p quad, n in block, 4 consecutive p)
    float* pB;        // [batch*H, L, N] per-head dB
    float* pC;        // [batch*H, L, N] per-head dC
    float *pA, *pD, *pbias;   // [batch*H] per-(batch, head) sums
    int64_t batch, L, H, G, N;
    int softplus;
    int in_bf16;
};
size_t m2_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t H, int64_t N);
void m2_bwd_carve(M2BwdArgs& a, void* ws);
// ssd: the chunked matrix form (bf16 inputs, N in {32, 64, 128}, 16-byte aligned
// x, z, dout, B, C); otherwise the recurrent form
hipError_t launch_m2_bwd(const M2BwdArgs& a, int in_bf16, int out_bf16, int ssd, hipStream_t stream);

// One-token state update (decoding), both variants.  Mamba-1: u, delta, z, y
// [batch, dim]; B, C [batch, N]; A [dim, N]; D, bias [dim]; state
// [batch, dim, N].  Mamba-2: u = x, z, y [batch, H, P]; delta = dt
// [batch, H]; B, C [batch, G, N]; A, D, bias [H]; state [batch, H, P, N].
struct StepArgs {
    const void* u;
    const void* delta;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* z;
    const float* bias;
    void* y;
    float* state;
    int64_t batch, dim;       // Mamba-1
    int64_t H, P, G;          // Mamba-2
    int N;
    int softplus;
    int vec;                  // A (16 bytes), B and C (4 elements) aligned for vector loads
};
hipError_t launch_step(const StepArgs& a, int in_bf16, int out_bf16, int mamba2, hipStream_t stream);

// Causal depthwise convolution: x, out [batch, dim, L]; w [dim, K]; bias [dim].
struct ConvArgs {
    const void* x;
    const float* w;
    const float* bias;
    void* out;
    int64_t batch, dim, L;
    int K;
    int silu;
    int vec_ok;   // L % 8 == 0 and 16-byte aligned rows of x and out
};
hipError_t launch_conv1d(const ConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream);
hipError_t launch_m2(const M2Args& a, int in_bf16, int out_bf16, hipStream_t stream);
// Chunked matrix (SSD) form on MFMA for bf16 inputs, P = 64, N in {64, 128}.
bool m2_ssd_supported(const M2Args& a, int in_bf16);
// ws: 1 = warp-specialised kernel (state waves and chunk waves), 0 = every wave in every phase
hipError_t launch_m2_ssd(const M2Args& a, int out_bf16, int ws, hipStream_t stream);

// Gated delta rule (q, k [batch, L, G, N]; v, y [batch, L, H, P]; g, beta
// [batch, L, H]; states [batch, H, P, N]).
struct DeltaArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const int32_t* lengths;   // tokens of each batch element, or NULL
    const float* h0;          // NULL = zero; the one-token update: last (in place)
    void* y;
    float* last;
    int64_t batch, L, H, P, G;
    int N;
    int NL;                   // chunked form: elements of a q or k row that are read (a multiple of 8),
    int64_t qk_row;           // and from one group's row to the next
    float scale;
    int vec;                  // token by token: rows of q, k and the states allow vector access
};
hipError_t launch_delta_rec(const DeltaArgs& a, int in_bf16, int out_bf16, hipStream_t stream);
// The chunked form: records of delta_record_bytes() for each of the
// batch x H x delta_chunks(L) chunks, then the scan over them.  Rows of q and
// k that are not made of aligned 16-byte pieces are copied first, padded to
// 64 or 128 elements (2 batch L G of them in `rows`; a is set to the copies).
int64_t delta_chunks(int64_t L);
size_t delta_record_bytes(bool grad);
hipError_t launch_delta_pad(DeltaArgs& a, int in_bf16, void* rows, hipStream_t stream);
hipError_t launch_delta_prep(const DeltaArgs& a, int in_bf16, bool grad, char* recs, hipStream_t stream);
hipError_t launch_delta_scan(const DeltaArgs& a, int in_bf16, int out_bf16, const char* recs, hipStream_t stream);

// Gradients of the gated delta rule; the arrays below dh0 are workspace
// (delta_bwd_carve).  f.y and f.last are unused.
struct DeltaBwdArgs {
    DeltaArgs f;
    const void* dout;
    const float* dlast;       // NULL = zero
    void *dq, *dk, *dv;
    float *dg, *dbeta, *dh0;
    char* recs;
    float* S;                 // [chunks, pad / 16, NP / 16, 64, 4] C tiles of the state entering each chunk
                              // (NP: N rounded up to 64 or 128)
    float* D;                 // the same of the adjoint of the state leaving it
    float* U;                 // [chunks, 64, pad]
    float* dR;                // [chunks, 64, pad]
    float *pq, *pk;           // [batch, L, H, N] per-head dq and dk when heads share q and k, else NULL
    int pad;                  // P rounded up to 32
    int vec_g;                // rows of dq and dk on 16-byte boundaries, N % 8 == 0
    int vec_p;                // rows of v and dout on 16-byte boundaries, P % 8 == 0
};
size_t delta_bwd_bytes(int64_t batch, int64_t L, int64_t H, int64_t G, int64_t P, int64_t N);
void delta_bwd_carve(DeltaBwdArgs& a, void* ws);
hipError_t launch_delta_keep(const DeltaArgs& a, int in_bf16, const char* recs, float* keep_s, float* keep_u, int pad,
                             hipStream_t stream);
hipError_t launch_delta_bwd(const DeltaBwdArgs& a, int in_bf16, int out_bf16, hipStream_t stream);

// Short causal convolution of token-major rows (x [batch, L, C], rows x_row
// and batch elements x_batch elements apart; weight [C, K]; states [batch,
// K - 1, C]).  y and dout are split into up to three dense tensors: channels
// from 0, begin[1], begin[2] on (begin[i] = C: no more pieces).
struct ShortConvArgs {
    const void* x;
    int64_t x_row, x_batch;
    const float* weight;
    const float* bias;        // NULL = 0
    const int32_t* lengths;   // tokens of each batch element, or NULL
    const void* state;        // NULL = zero
    void* y[3];
    void* last;               // the state after; one token: the state, in place
    const void* dout[3];
    const void* dlast;        // NULL = zero
    void* dx;
    void* dstate;             // NULL = skip
    float *dweight, *dbias;   // NULL = skip
    float* part;              // [batch run_blocks, K + 1, C] sums of the taps' and the bias' gradients
    int64_t begin[3];
    int64_t batch, L, C;
    int K, silu;
    int V, cols;              // short_conv_plan: channels a thread, columns a workgroup,
    int64_t run, col_blocks, run_blocks;   // tokens a run, workgroups over the channels and over the tokens
};
void short_conv_plan(ShortConvArgs& a, bool bwd);
hipError_t launch_short_conv_fwd(const ShortConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream);
hipError_t launch_short_conv_bwd(const ShortConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream);
hipError_t launch_short_conv_step(const ShortConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream);

// Sums of the columns of n partial rows of n0 + n1 fp32: the first n0 to out0,
// the others to out1 (NULL = skip).  `part` has column_sums_rows(n) rows.
int64_t column_sums_rows(int64_t n);
hipError_t launch_column_sums(float* part, int64_t n, int64_t n0, int64_t n1, float* out0, float* out1, hipStream_t stream);

// Mamba-2 with the short convolution in front (xbc [batch, L, H P + 2 G N], dt
// [batch, L, H], strided; y [batch, L, H, P] dense; states [batch, H, P, N]
// fp32 and [batch, K - 1, H P + 2 G N]).
struct M2ConvArgs {
    ShortConvArgs conv;       // of xbc; y unused
    const void* dt;
    int64_t dt_row, dt_batch;
    const float* A;
    const float* D;           // NULL = 0
    const float* dt_bias;     // NULL = 0
    const float* h0;          // NULL = zero
    void* y;
    float* last;              // NULL = skip; one token: the state, in place
    int64_t batch, L, H, P, G, N;
};
// The sequence forms and the bytes of workspace they need: token by token, and
// in 64-token chunks (np: N rounded up to 32, 64 or 128).
size_t m2_rec_bytes(const M2ConvArgs& a);
hipError_t launch_m2_rec(const M2ConvArgs& a, int in_bf16, int out_bf16, void* ws, hipStream_t stream);
size_t m2_chunk_bytes(const M2ConvArgs& a, int in_bf16);
hipError_t launch_m2_chunk(const M2ConvArgs& a, int in_bf16, int out_bf16, void* ws, hipStream_t stream);
hipError_t launch_m2_prep(const M2ConvArgs& a, int in_bf16, int out_bf16, int np, char* recs, int64_t chunks, hipStream_t stream);
hipError_t launch_m2_conv_step(const M2ConvArgs& a, int in_bf16, int out_bf16, hipStream_t stream);

// RMS norm of s = x + residual, or s = x silu(gate), over the groups of a row.
struct RmsArgs {
    const void* x;            // forward: x; gradients: dy
    const void* res;          // forward: residual or NULL; gradients: s, or x where there is a gate
    const void* gate;         // rows gate_row elements apart, or NULL
    const float* weight;      // NULL = 1
    const float* rstd_in;     // gradients: [rows, groups]
    const void* dres_in;      // gradients: of s from its other uses, or NULL
    void* y;                  // forward: y; gradients: dx
    void* res_out;            // forward: s; gradients: dresidual
    void* dgate;
    float* rstd;
    float* scale;             // forward in 8 bits: [rows, blocks of a row]
    float* dweight;
    float* part;              // gradients: [blocks, dim] partial sums of dweight, and room to add them up
    int64_t rows, dim, gate_row, groups, width;   // width: of a group, dim / groups
    int64_t block, row_blocks;   // elements to a scale, scales to a row
    int blocks;               // gradients: workgroups to a group
    float eps, inv_width;
};
size_t rms_bwd_part_bytes(int64_t rows, int64_t dim, int64_t groups);
int rms_bwd_blocks(int64_t rows, int64_t width);
bool rms_reads_again(int64_t width);   // dweight by a kernel of its own, behind the other gradients
hipError_t launch_rms_fwd(const RmsArgs& a, int in_bf16, int res_bf16, int out_dtype, hipStream_t stream);
hipError_t launch_rms_bwd(const RmsArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t stream);

// Layer norm with dropout and residual sum in front.
struct NormArgs {
    const void* x;            // forward: x; gradients: dy
    const void* res;          // forward: residual; gradients: s
    const float* weight;
    const float* bias;
    const float* mean_in;     // gradients
    const float* rstd_in;
    const void* dres_in;
    void* y;                  // forward: y; gradients: dx
    void* res_out;            // forward: s; gradients: dresidual
    float* mean;
    float* rstd;
    float* dweight;
    float* dbias;
    float* part;              // gradients: [blocks, 2, dim] partial sums of dweight, dbias, and room to add them up
    int64_t rows, dim;
    int blocks;
    float eps, inv_dim;
    uint64_t seed, offset;
    uint64_t keep_from;       // a word below this drops its element (2^32: all are dropped)
    float keep_scale;
    int drop;                 // dropout is on
    int vec;                  // rows start on 16-byte boundaries, dim % 8 == 0
};
int norm_bwd_blocks(int64_t rows, int64_t dim);
size_t norm_bwd_part_bytes(int64_t rows, int64_t dim);
hipError_t launch_norm_fwd(const NormArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs& a, int in_bf16, int res_bf16, int out_bf16, hipStream_t stream);

struct DropArgs {
    const void* x;
    void* y;
    int64_t n;
    uint64_t seed, offset, keep_from;
    float keep_scale;
    int vec;                  // x and y on 16-byte boundaries
};
hipError_t launch_dropout(const DropArgs& a, int bf16, hipStream_t stream);

}  // namespace selscan
