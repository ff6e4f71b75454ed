/*
 * selscan.h -- C ABI of libselscan, the selective state-space scan of Mamba
 * on AMD Instinct MI355X (gfx950).
 *
 * What is computed.  For every batch b, channel d, state index n and token t
 * (Mamba-1 form):
 *
 *     Delta_t  = softplus(delta_t + delta_bias_d)      (or delta_t + bias if softplus == 0)
 *     h_t[n]   = exp(Delta_t * A[d,n]) * h_{t-1}[n] + Delta_t * B_t[n] * u_t,   h_{-1} = 0
 *     y_t      = (sum_n C_t[n] * h_t[n] + D_d * u_t) * silu(z_t)             (gate optional)
 *
 * Sources: the "Understanding Mamba and Selective State Space Models (SSMs)"
 * blog, section 2.2 (the selective update with exp(Delta A), the recurrent
 * scan from a zero state, softplus keeping Delta positive) and section 2.1
 * (the read-out y = C h + D x); the Mamba README on the gittoolsai page for
 * state-spaces/mamba, sections "Selective SSM" (the layer), "Mamba-2" and
 * "Initialization" (the Delta bias); the "model-architecture-mamba" skill
 * page (Mamba-2: multi-head, d_state 128, headdim 64).  Where the pages are
 * silent the plainest reading is taken: the read-out sums over n, the gate
 * multiplies the D term too, the initial state is zero, A is stored negative.
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are DEVICE pointers owned by the caller, dense and
 *    row-major in the layouts given below (but for rows whose strides a shape
 *    names).  The library keeps no pointer after
 *    a call returns.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Work
 *    is enqueued on it and the call returns without synchronising.  Faults
 *    inside a kernel surface at the caller's next synchronisation.
 *  - Argument errors are detected on the host before any device work and
 *    return SELSCAN_ERR_INVALID_ARG / SELSCAN_ERR_UNSUPPORTED with a message
 *    available from selscan_last_error() on the calling thread.  No C++
 *    exception crosses this interface; the library never aborts the process.
 *  - NaN and Inf in the inputs propagate to the outputs; nothing is clamped.
 *  - Calls on distinct streams may run concurrently.
 */
#ifndef SELSCAN_H
#define SELSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SELSCAN_OK = 0,
    SELSCAN_ERR_INVALID_ARG = 1,  /* null required pointer, bad size, overflow */
    SELSCAN_ERR_UNSUPPORTED = 2,  /* valid but not implemented (dtype, d_state) */
    SELSCAN_ERR_NO_DEVICE = 3,    /* no usable gfx950 device */
    SELSCAN_ERR_LAUNCH = 4,       /* the HIP runtime refused a launch or an allocation */
    SELSCAN_ERR_WORKSPACE = 5     /* caller workspace smaller than selscan_*_workspace_bytes */
} selscan_status_t;

typedef enum {
    SELSCAN_F32 = 0,   /* IEEE binary32 */
    SELSCAN_BF16 = 1,  /* bfloat16 (upper half of a binary32); stores round to nearest even */
    SELSCAN_E4M3 = 2   /* 8 bits, OCP e4m3 without infinities: an output of selscan_rms_norm_fwd alone */
} selscan_dtype_t;

/*
 * Mamba-1 problem description.
 *   batch  B >= 1, dim D >= 1 (channels, d_inner), dstate N in {1..16},
 *   1 <= seqlen L < 16777216 (2^24; UNSUPPORTED from 2^24 on).
 *   in_dtype : dtype of u, delta, z, B, C.
 *   out_dtype: dtype of y.
 *   workspace: optional device scratch of at least selscan_workspace_bytes()
 *              bytes, 256-byte aligned.  NULL: the library allocates what it
 *              needs with stream-ordered hipMallocAsync / hipFreeAsync on the
 *              call's stream.
 */
typedef struct {
    int64_t batch, dim, dstate, seqlen;
    int32_t in_dtype;
    int32_t out_dtype;
    void* workspace;
    size_t workspace_bytes;
} selscan_shape_t;

/* Bytes of workspace selscan_fwd needs for `shape` (0 if none). */
size_t selscan_workspace_bytes(const selscan_shape_t* shape);

/*
 * Mamba-1 selective scan (the selective SSM layer of the Mamba README; the
 * update of section 2.2 of the "Understanding Mamba ..." blog).
 *
 *   u          [B, D, L]  in_dtype   input x_t of each channel
 *   delta      [B, D, L]  in_dtype   Delta pre-activation
 *   A          [D, N]     fp32       state matrix diagonal (normally < 0)
 *   B          [B, N, L]  in_dtype   input projection, shared by all channels
 *   C          [B, N, L]  in_dtype   output projection, shared by all channels
 *   D          [D]        fp32       skip weight; NULL = no skip term
 *   z          [B, D, L]  in_dtype   gate; NULL = no silu(z) gating
 *   delta_bias [D]        fp32       added to delta before softplus; NULL = 0
 *   softplus   0 or 1     apply softplus to delta + bias
 *   y          [B, D, L]  out_dtype  output (written)
 *   last_state [B, D, N]  fp32       h after the last token (written); NULL = skip
 *
 * Returns SELSCAN_OK once the work is enqueued.
 */
selscan_status_t selscan_fwd(const selscan_shape_t* shape,
                             const void* u, const void* delta, const float* A,
                             const void* B, const void* C, const float* D,
                             const void* z, const float* delta_bias, int softplus,
                             void* y, float* last_state, void* stream);

/*
 * selscan_fwd from a given initial state instead of zero: the scan continues
 * a sequence whose state after its previous part is h0 (the recurrence of
 * section 2.2 of the "Understanding Mamba ..." blog, resumed; the streaming
 * use on the tutorial and skill pages).
 *   h0 [B, D, N] fp32 device memory, read only; NULL = zero state (then
 *      identical to selscan_fwd).  h0 and last_state must not alias: chunks
 *      of one channel run concurrently.
 * Other arguments, errors and workspace as for selscan_fwd.
 */
selscan_status_t selscan_fwd_h0(const selscan_shape_t* shape,
                                const void* u, const void* delta, const float* A,
                                const void* B, const void* C, const float* D,
                                const void* z, const float* delta_bias, int softplus,
                                const float* h0, void* y, float* last_state, void* stream);

/*
 * selscan_fwd_h0 for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * It allocates nothing (no hipMalloc, hipFree or allocating library call):
 * its scratch is a file-scope device array of SELSCAN_NOALLOC_SCRATCH_BYTES
 * (64 MiB) that each GPU the library runs on holds until the process ends.
 *   shape      as for selscan_fwd; its workspace fields are ignored.
 *   other arguments as for selscan_fwd_h0 (h0 NULL = zero state).
 * Errors as for selscan_fwd_h0, plus SELSCAN_ERR_WORKSPACE when the shape
 * needs more scratch than the maximum (selscan_workspace_bytes(shape) >
 * SELSCAN_NOALLOC_SCRATCH_BYTES; e.g. batch 1, dim 2048, L 2^20 needs
 * ~137 MB), before any device work.  Every call on one GPU shares that GPU's
 * array: calls that overlap on one GPU (concurrent streams without ordering
 * between them) race and must not be issued.  Device ids >= 64 are
 * UNSUPPORTED.
 */
#define SELSCAN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
selscan_status_t selscan_fwd_noalloc(const selscan_shape_t* shape,
                                     const void* u, const void* delta, const float* A,
                                     const void* B, const void* C, const float* D,
                                     const void* z, const float* delta_bias, int softplus,
                                     const float* h0, void* y, float* last_state, void* stream);

/*
 * One-token state update (decoding; the recurrent view of section 2.2 of the
 * "Understanding Mamba ..." blog, one token at a time as the tutorial and
 * skill pages use it for generation).  shape: batch, dim, dstate N (1..16),
 * in_dtype, out_dtype; seqlen, workspace and workspace_bytes are ignored.
 *   state      [B, D, N] fp32  h before the token on entry, after it on
 *                              return (updated in place); 16-byte aligned
 *                              when N is a multiple of 4
 *   u, delta   [B, D]    in_dtype
 *   A          [D, N]    fp32
 *   B, C       [B, N]    in_dtype   this token's projections
 *   D, delta_bias [D]    fp32       NULL = 0
 *   z          [B, D]    in_dtype   NULL = no gate
 *   y          [B, D]    out_dtype  (written)
 * No workspace.  Errors as for selscan_fwd; UNSUPPORTED for N > 16.
 */
selscan_status_t selscan_step(const selscan_shape_t* shape, float* state,
                              const void* u, const void* delta, const float* A,
                              const void* B, const void* C, const float* D,
                              const void* z, const float* delta_bias, int softplus,
                              void* y, void* stream);

/* Bytes of workspace selscan_bwd needs for `shape` (0 on a bad shape). */
size_t selscan_bwd_workspace_bytes(const selscan_shape_t* shape);

/*
 * Gradients of the Mamba-1 scan (training; reverse mode through the
 * recurrence of section 2.2 of the "Understanding Mamba ..." blog, the layer
 * the Mamba README trains end to end).  For out = selscan_fwd_h0(...) and
 * dout = d loss / d out, writes the gradient of the loss with respect to
 * every input.  The states are recomputed from the inputs (nothing from the
 * forward call is needed).
 *   u .. softplus, h0   as for selscan_fwd_h0 (h0 NULL = zero state)
 *   dout        [B, D, L]  out_dtype   gradient of the output
 *   du, ddelta  [B, D, L]  fp32        (written); ddelta is with respect to
 *                                      delta itself (before bias/softplus)
 *   dA          [D, N]     fp32        (written)
 *   dB, dC      [B, N, L]  fp32        (written)
 *   dD          [D]        fp32        (written; NULL = skip; 0 when D is NULL)
 *   dz          [B, D, L]  fp32        (written; required when z is given,
 *                                      ignored otherwise)
 *   ddelta_bias [D]        fp32        (written; NULL = skip)
 *   dh0         [B, D, N]  fp32        (written; NULL = skip)
 * seqlen <= 4194304 (2^22; UNSUPPORTED above).
 * Gradients must not alias inputs or each other.  Sums over channels,
 * batches and time are taken in a fixed order: results are reproducible
 * bit for bit.  shape->workspace as for selscan_fwd, sized by
 * selscan_bwd_workspace_bytes.  Errors as for selscan_fwd, plus
 * SELSCAN_ERR_INVALID_ARG for a NULL required gradient.
 */
selscan_status_t selscan_bwd(const selscan_shape_t* shape,
                             const void* u, const void* delta, const float* A,
                             const void* B, const void* C, const float* D,
                             const void* z, const float* delta_bias, int softplus,
                             const float* h0, const void* dout,
                             float* du, float* ddelta, float* dA, float* dB, float* dC,
                             float* dD, float* dz, float* ddelta_bias, float* dh0,
                             void* stream);

/*
 * Mamba-2 problem description.
 *   batch >= 1, seqlen >= 1, nheads H >= 1, headdim P >= 1, ngroups G >= 1
 *   with H % G == 0, dstate N in {16, 32, 64, 128}.
 *   in_dtype: dtype of x, dt, z, B, C; out_dtype: dtype of y.
 *   workspace: as for selscan_shape_t.
 */
typedef struct {
    int64_t batch, seqlen, nheads, headdim, ngroups, dstate;
    int32_t in_dtype;
    int32_t out_dtype;
    void* workspace;
    size_t workspace_bytes;
} selscan_m2_shape_t;

size_t selscan_mamba2_workspace_bytes(const selscan_m2_shape_t* shape);

/*
 * Mamba-2 multi-head selective scan (the Mamba-2 block of the Mamba README;
 * the "model-architecture-mamba" page's multi-head Mamba-2): a scalar A per
 * head, one Delta per (batch, token, head) shared by the head's P channels,
 * B and C shared by the heads of a group; head h reads group h / (H / G).
 *
 *   x          [B, L, H, P]  in_dtype
 *   dt         [B, L, H]     in_dtype   Delta pre-activation
 *   A          [H]           fp32
 *   B, C       [B, L, G, N]  in_dtype
 *   D          [H]           fp32       NULL = no skip
 *   z          [B, L, H, P]  in_dtype   NULL = no gate
 *   dt_bias    [H]           fp32       NULL = 0
 *   y          [B, L, H, P]  out_dtype  (written)
 *   last_state [B, H, P, N]  fp32       (written); NULL = skip
 *
 * Two forms compute it.  bf16 inputs with P = 64, N in {64, 128} and x, B, C
 * on 16-byte boundaries take the chunked matrix form named in the README's
 * Mamba-2 section (64-token chunks, the products on the matrix cores in bf16
 * with fp32 accumulation; the fp32 operands -- the intra-chunk matrix, the
 * state and the weighted x -- enter as bf16 pairs, relative error near
 * 2^-16, and sums run in another order than the recurrence's); every other
 * shape takes the recurrent form in fp32 (whose chunk carries on long
 * sequences are what selscan_mamba2_workspace_bytes sizes).
 */
selscan_status_t selscan_mamba2_fwd(const selscan_m2_shape_t* shape,
                                    const void* x, const void* dt, const float* A,
                                    const void* B, const void* C, const float* D,
                                    const void* z, const float* dt_bias, int softplus,
                                    void* y, float* last_state, void* stream);

/* selscan_mamba2_fwd from an initial state h0 [B, H, P, N] fp32 (NULL =
 * zero); h0 and last_state must not alias. */
selscan_status_t selscan_mamba2_fwd_h0(const selscan_m2_shape_t* shape,
                                       const void* x, const void* dt, const float* A,
                                       const void* B, const void* C, const float* D,
                                       const void* z, const float* dt_bias, int softplus,
                                       const float* h0, void* y, float* last_state, void* stream);

/* Bytes of workspace selscan_mamba2_bwd needs for `shape` (0 on a bad
 * shape): per (batch, head) the state entering every 8-token tile
 * (64 x N fp32 each, i.e. 4 KiB per token and head at N = 128; the chunked
 * form below uses one state per 32 tokens of this space) and the head's
 * share of dB and dC (2 x L x N fp32).  It grows with batch x seqlen x
 * nheads: 5.4 GB for batch 8, seqlen 4096, 32 heads. */
size_t selscan_mamba2_bwd_workspace_bytes(const selscan_m2_shape_t* shape);

/*
 * Gradients of the Mamba-2 scan (training; reverse mode through the
 * multi-head recurrence of the README's "Mamba-2" section: one scalar decay
 * per token and head, B and C shared by the heads of a group).  For
 * out = selscan_mamba2_fwd_h0(...) and dout = d loss / d out, writes the
 * gradient of the loss with respect to every input; the states are
 * recomputed from the inputs.  bf16 inputs with N >= 32 and 16-byte aligned
 * x, z, dout, B, C take the chunked matrix form (32-token chunks, products
 * on the matrix cores with fp32 operands split into bf16 hi + lo pairs, the
 * state entering each chunk kept in the workspace; the environment variable
 * SELSCAN_M2_BWD_SSD=0 turns it off); other calls take the recurrent form
 * (fp32, the state entering every 8-token tile kept).
 *   x .. softplus, h0   as for selscan_mamba2_fwd_h0 (h0 NULL = zero state)
 *   dout        [B, L, H, P]  out_dtype   gradient of the output
 *   dx          [B, L, H, P]  fp32        (written)
 *   ddt         [B, L, H]     fp32        (written; with respect to dt itself,
 *                                         before bias and softplus)
 *   dA          [H]           fp32        (written)
 *   dB, dC      [B, L, G, N]  fp32        (written; summed over the heads of
 *                                         each group and their channels)
 *   dD          [H]           fp32        (written; NULL = skip; 0 when D is NULL)
 *   dz          [B, L, H, P]  fp32        (written; required when z is given,
 *                                         ignored otherwise)
 *   ddt_bias    [H]           fp32        (written; NULL = skip; 0 when dt_bias
 *                                         is NULL)
 *   dh0         [B, H, P, N]  fp32        (written; NULL = skip)
 * headdim P = 64 only (SELSCAN_ERR_UNSUPPORTED otherwise); N in
 * {16, 32, 64, 128}.  One workgroup per (batch, head) walks the whole
 * sequence: time is not split, so few (batch, head) units leave most of the
 * GPU idle.  Gradients must not alias inputs or each other.  Sums
 * over heads, channels, batches and time run in a fixed order: results are
 * reproducible bit for bit.  shape->workspace as for selscan_mamba2_fwd,
 * sized by selscan_mamba2_bwd_workspace_bytes.  Errors as for
 * selscan_mamba2_fwd, plus SELSCAN_ERR_INVALID_ARG for a NULL required
 * gradient.
 */
selscan_status_t selscan_mamba2_bwd(const selscan_m2_shape_t* shape,
                                    const void* x, const void* dt, const float* A,
                                    const void* B, const void* C, const float* D,
                                    const void* z, const float* dt_bias, int softplus,
                                    const float* h0, const void* dout,
                                    float* dx, float* ddt, float* dA, float* dB, float* dC,
                                    float* dD, float* dz, float* ddt_bias, float* dh0,
                                    void* stream);

/*
 * Mamba-2 one-token update.  shape: batch, nheads H, headdim P, ngroups G,
 * dstate N in {16, 32, 64, 128}, dtypes; seqlen and workspace ignored.
 *   state   [B, H, P, N] fp32  updated in place, 16-byte aligned
 *   x, z    [B, H, P]    in_dtype (z NULL = no gate)
 *   dt      [B, H]       in_dtype
 *   A, D, dt_bias [H]    fp32 (D, dt_bias NULL = 0)
 *   B, C    [B, G, N]    in_dtype
 *   y       [B, H, P]    out_dtype (written)
 */
selscan_status_t selscan_mamba2_step(const selscan_m2_shape_t* shape, float* state,
                                     const void* x, const void* dt, const float* A,
                                     const void* B, const void* C, const float* D,
                                     const void* z, const float* dt_bias, int softplus,
                                     void* y, void* stream);

/*
 * Causal depthwise convolution ahead of the scan (section 3.3 of the
 * "Understanding Mamba ..." blog: a width-4 convolution whose output at a
 * token sees it and the three before it; the README's causal-conv1d layer):
 *   out[b,d,t] = act(bias[d] + sum_{k<K} weight[d,k] x[b,d,t-(K-1)+k]),
 * x before the first token taken as zero, act = silu when silu == 1, else
 * identity.  weight[d, K-1] multiplies the current token.
 *   x       [B, D, L]  in_dtype
 *   weight  [D, K]     fp32
 *   bias    [D]        fp32, NULL = 0
 *   out     [B, D, L]  out_dtype (written; must not alias x)
 * width K in 1..64 (UNSUPPORTED above); no workspace; asynchronous on stream.
 */
typedef struct {
    int64_t batch, dim, seqlen, width;
    int32_t in_dtype, out_dtype;
} selscan_conv_shape_t;

selscan_status_t selscan_conv1d(const selscan_conv_shape_t* shape, const void* x,
                                const float* weight, const float* bias, int silu,
                                void* out, void* stream);

/*
 * Gated delta rule: the recurrence next to the Mamba-2 scan whose heads erase
 * along the current key before they write.  Tensors and state are laid out as
 * for the Mamba-2 scan, with selscan_m2_shape_t's dstate N the size of a key
 * and headdim P the size of a value.  For every batch element and head, with
 * S [P, N] and S_{-1} = h0 (zero when NULL):
 *
 *     S_t = exp(g_t) (S_{t-1} - beta_t (S_{t-1} k_t) k_t^T) + beta_t v_t k_t^T
 *     y_t = scale S_t q_t
 *
 *   q, k       [B, L, G, N]  in_dtype   shared by the heads of a group: head h
 *                                       reads group h / (H / G); taken as
 *                                       given (normalise k before the call)
 *   v          [B, L, H, P]  in_dtype
 *   g          [B, L, H]     fp32       log decay, normally <= 0; minus infinity
 *                                       (or -200 and less) is a decay of zero
 *   beta       [B, L, H]     fp32       write strength, normally in (0, 1)
 *   lengths    [B]           int32      tokens of each batch element, device
 *                                       memory, clamped to 0..L; NULL = L.
 *                                       Tokens past the end are not read,
 *                                       their y is zero, and last_state is
 *                                       the state after the last token inside
 *   h0         [B, H, P, N]  fp32       NULL = zero
 *   y          [B, L, H, P]  out_dtype  (written)
 *   last_state [B, H, P, N]  fp32       (written; NULL = skip); may not alias h0
 *
 * 1 <= N <= 128, H P <= 2^22, G <= 2^15 (UNSUPPORTED above), any L.  State,
 * decays and sums are fp32, and so are products in effect, whatever the types
 * of inputs and outputs: what is written in bf16 is the fp32 result, rounded
 * once.  Past 16 tokens the sequence is worked on in
 * chunks of 64, as matrix products: a NaN or infinity in a token reaches every
 * y of its chunk and head, and what follows.
 *
 * Workspace as for the other entry points, sized by
 * selscan_delta_workspace_bytes: per head and 64 tokens 32 KB, and where N is
 * no multiple of 8 padded copies of q and k (which are
 * allocated on `stream` by the call itself where only their addresses are off
 * a 16-byte boundary).
 */
size_t selscan_delta_workspace_bytes(const selscan_m2_shape_t* shape);

selscan_status_t selscan_delta_fwd(const selscan_m2_shape_t* shape,
                                   const void* q, const void* k, const void* v,
                                   const float* g, const float* beta, float scale,
                                   const int32_t* lengths, const float* h0,
                                   void* y, float* last_state, void* stream);

/* Bytes of workspace selscan_delta_bwd needs for `shape` (0 on a bad shape).
 * It grows with batch x heads x L: per head and 64 tokens two states, two
 * P-wide rows per token and 57.6 KB (254 KB in all at N = P = 128; 521 MB for
 * batch 4, L 2048, 16 heads), and 2 N fp32 per token and head where heads
 * share q and k. */
size_t selscan_delta_bwd_workspace_bytes(const selscan_m2_shape_t* shape);

/*
 * Gradients of the gated delta rule (training; reverse mode through the
 * recurrence, the states recomputed from the inputs).
 *   q .. lengths, h0  as for selscan_delta_fwd
 *   dout         [B, L, H, P]  out_dtype  gradient of y (not read past a
 *                                         sequence's end)
 *   dlast_state  [B, H, P, N]  fp32       gradient of last_state; NULL = 0
 *   dq, dk       [B, L, G, N]  in_dtype   (written; summed over the heads of a
 *                                         group in fp32, then rounded once)
 *   dv           [B, L, H, P]  in_dtype   (written)
 *   dg, dbeta    [B, L, H]     fp32       (written)
 *   dh0          [B, H, P, N]  fp32       (written; NULL = skip)
 * Gradients of tokens past a sequence's end are zero.  Gradients must not
 * alias inputs or each other.  Sums run in a fixed order: results are
 * reproducible bit for bit.  Unlike the scans' gradients, dq, dk and dv come
 * in the inputs' type: they are read next by the backward of a projection.
 */
selscan_status_t selscan_delta_bwd(const selscan_m2_shape_t* shape,
                                   const void* q, const void* k, const void* v,
                                   const float* g, const float* beta, float scale,
                                   const int32_t* lengths, const float* h0,
                                   const void* dout, const float* dlast_state,
                                   void* dq, void* dk, void* dv, float* dg, float* dbeta,
                                   float* dh0, void* stream);

/*
 * Gated delta rule, one token: shape as for selscan_delta_fwd (seqlen and
 * workspace ignored); q, k [B, G, N], v [B, H, P] in_dtype, g, beta [B, H]
 * fp32, y [B, H, P] out_dtype.  state [B, H, P, N] fp32 is updated in place
 * (16-byte aligned when N is a multiple of 4).
 */
selscan_status_t selscan_delta_step(const selscan_m2_shape_t* shape, float* state,
                                    const void* q, const void* k, const void* v,
                                    const float* g, const float* beta, float scale,
                                    void* y, void* stream);

/*
 * Dropout whose mask is a function of (seed, offset, element index) and is
 * never stored: element i is kept when word i % 4 of Philox4x32-10 (Salmon,
 * Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)
 * at counter (i / 4, offset) -- i / 4 in words 0 and 1, offset in words 2 and
 * 3, low halves first -- and key `seed` is at least floor(p 2^32).  Kept
 * elements are multiplied by 1 / (1 - p), the others are zero whatever they
 * were.  The gradient is the same call on the output's gradient.
 *   x, y  [n]  dtype   y may be x; n >= 1, 0 <= p <= 1
 */
typedef struct {
    int64_t n;
    int32_t dtype;
    double p;
    uint64_t seed, offset;
} selscan_dropout_shape_t;

selscan_status_t selscan_dropout(const selscan_dropout_shape_t* shape, const void* x, void* y, void* stream);

/*
 * Layer norm between two blocks, with the dropout and the residual sum that
 * come before it:
 *
 *     s    = dropout(x) + residual            (element r * dim + d of the mask)
 *     mean = sum_d s / dim;  rstd = 1 / sqrt(sum_d (s - mean)^2 / dim + eps)
 *     y    = (s - mean) rstd weight + bias
 *
 *   x            [rows, dim]  in_dtype
 *   residual     [rows, dim]  res_dtype   NULL = 0
 *   weight, bias [dim]        fp32        NULL = 1 and 0
 *   y            [rows, dim]  out_dtype   (written); may be x where their types agree
 *   residual_out [rows, dim]  res_dtype   s (written; NULL = skip); may be residual
 *   mean, rstd   [rows]       fp32        (written; NULL = skip)
 * p, seed, offset as for selscan_dropout; p = 0 leaves x as it is.  The sums
 * are fp32 over s before it is rounded to res_dtype.  rows, dim >= 1;
 * workspace is used by the gradients only.
 */
typedef struct {
    int64_t rows, dim;
    int32_t in_dtype, res_dtype, out_dtype;
    float eps;
    double p;
    uint64_t seed, offset;
    void* workspace;
    size_t workspace_bytes;
} selscan_norm_shape_t;

selscan_status_t selscan_layer_norm_fwd(const selscan_norm_shape_t* shape, const void* x, const void* residual,
                                        const float* weight, const float* bias, void* y, void* residual_out,
                                        float* mean, float* rstd, void* stream);

/* Bytes of workspace selscan_layer_norm_bwd needs (0 on a bad shape). */
size_t selscan_layer_norm_bwd_workspace_bytes(const selscan_norm_shape_t* shape);

/*
 * Gradients of selscan_layer_norm_fwd from what it kept (s as written to
 * residual_out -- or x itself when there was neither dropout nor residual --
 * mean and rstd):
 *
 *     xhat = (s - mean) rstd;  w = dy weight
 *     ds   = rstd (w - sum_d w / dim - xhat sum_d (w xhat) / dim) + dresidual_out
 *     dx   = dropout's gradient of ds;  dresidual = ds
 *     dweight = sum_r dy xhat;  dbias = sum_r dy
 *
 *   dy            [rows, dim]  out_dtype
 *   s             [rows, dim]  res_dtype
 *   weight        [dim]        fp32        NULL = 1
 *   mean, rstd    [rows]       fp32
 *   dresidual_out [rows, dim]  res_dtype   gradient of s from its other uses; NULL = 0
 *   dx            [rows, dim]  in_dtype    (written; NULL = skip)
 *   dresidual     [rows, dim]  res_dtype   (written; NULL = skip); may be dresidual_out
 *   dweight, dbias [dim]       fp32        (written; NULL = skip)
 * Sums over rows run in a fixed order: results are reproducible bit for bit.
 * Workspace as for the other entry points.
 */
selscan_status_t selscan_layer_norm_bwd(const selscan_norm_shape_t* shape, const void* dy, const void* s,
                                        const float* weight, const float* mean, const float* rstd,
                                        const void* dresidual_out, void* dx, void* dresidual,
                                        float* dweight, float* dbias, void* stream);

/*
 * Short causal convolution of token-major rows, as the mixers take it in front
 * of their scan: width K in 2..4 (UNSUPPORTED otherwise; selscan_conv1d has
 * longer ones), rows read where a projection left them, the tokens before the
 * first from a state, padded batches.  Per batch element b and channel d:
 *
 *     pre_t = bias[d] + sum_{k<K} weight[d,k] x[b,t-(K-1)+k,d]
 *     out_t = pre_t sigmoid(pre_t) when silu == 1, else pre_t
 *
 * shape: x has seqlen rows of dim elements, a row x_row and a batch element
 * x_batch elements after the one before (0 and more; any address of an
 * element).  split: the outputs' channels, in order (dim in all); split[1] =
 * split[2] = 0 for one output.
 *   x          [B, L, D]     in_dtype   strided as above
 *   weight     [D, K]        fp32
 *   bias       [D]           fp32       NULL = 0
 *   lengths    [B]           int32      as for selscan_delta_fwd: tokens past
 *                                       the end are not read, their out is zero
 *   state      [B, K-1, D]   in_dtype   the K - 1 tokens before the first,
 *                                       oldest first; NULL = zero
 *   y0, y1, y2 [B, L, split[i]] out_dtype (written; NULL where split[i] is 0)
 *   last_state [B, K-1, D]   in_dtype   the last K - 1 tokens inside the
 *                                       sequence, of `state` and x (written;
 *                                       NULL = skip); may not alias state
 * Sums and the activation are fp32.  Outputs must not overlap inputs or each
 * other (INVALID_ARG).  No workspace (the field is the gradients').
 */
typedef struct {
    int64_t batch, seqlen, dim, width;
    int64_t x_row, x_batch;
    int64_t split[3];
    int32_t in_dtype, out_dtype;
    void* workspace;
    size_t workspace_bytes;
} selscan_short_conv_shape_t;

selscan_status_t selscan_short_conv_fwd(const selscan_short_conv_shape_t* shape, const void* x, const float* weight,
                                        const float* bias, int silu, const int32_t* lengths, const void* state,
                                        void* y0, void* y1, void* y2, void* last_state, void* stream);

/* Bytes of workspace selscan_short_conv_bwd needs (0 on a bad shape). */
size_t selscan_short_conv_bwd_workspace_bytes(const selscan_short_conv_shape_t* shape);

/*
 * Gradients of selscan_short_conv_fwd; what the activation needs is made again
 * from x.
 *   x .. state           as for selscan_short_conv_fwd
 *   dout0, dout1, dout2  [B, L, split[i]]  out_dtype   gradients of y0, y1, y2
 *                                          (not read past a sequence's end)
 *   dlast_state          [B, K-1, D]       in_dtype    gradient of last_state; NULL = 0
 *   dx                   [B, L, D]         in_dtype    (written; dense; zero past the end)
 *   dweight              [D, K]            fp32        (written; NULL = skip)
 *   dbias                [D]               fp32        (written; NULL = skip)
 *   dstate               [B, K-1, D]       in_dtype    (written; NULL = skip)
 * Gradients must not overlap inputs or each other (INVALID_ARG).  Sums run in a
 * fixed order: results are reproducible bit for bit.  Workspace as for the other
 * entry points; none where dweight and dbias are NULL.
 */
selscan_status_t selscan_short_conv_bwd(const selscan_short_conv_shape_t* shape, const void* x, const float* weight,
                                        const float* bias, int silu, const int32_t* lengths, const void* state,
                                        const void* dout0, const void* dout1, const void* dout2,
                                        const void* dlast_state, void* dx, float* dweight, float* dbias, void* dstate,
                                        void* stream);

/* One token: x [B, D] (batch elements x_batch apart; seqlen, x_row and split
 * ignored), y [B, D] out_dtype; state [B, K-1, D] in_dtype moves on in place.
 * y may be x where their types agree and x is dense; otherwise y and state must
 * not overlap x or each other (INVALID_ARG). */
selscan_status_t selscan_short_conv_step(const selscan_short_conv_shape_t* shape, void* state, const void* x,
                                         const float* weight, const float* bias, int silu, void* y, void* stream);

/*
 * Mamba-2 mixer between its projections, for prompts: the short convolution
 * with silu over xbc = (x, B, C), softplus of dt + dt_bias, and the Mamba-2
 * scan, in one call; the convolution's result is not rounded to 16 bits on the
 * way.  With v = silu(conv(xbc)) (selscan_short_conv_fwd) and x, B, C its
 * channels in that order:
 *
 *     Delta_t = softplus(dt_t + dt_bias[h])
 *     S_t = exp(Delta_t A[h]) S_{t-1} + Delta_t x_t B_t^T,  S_{-1} = h0
 *     y_t = S_t C_t + D[h] x_t
 *
 *   xbc         [B, L, H P + 2 G N]  in_dtype   rows xbc_row, batch elements
 *                                               xbc_batch elements apart
 *   dt          [B, L, H]            in_dtype   the same with dt_row, dt_batch
 *   conv_weight [H P + 2 G N, K]     fp32       K in 2..4
 *   conv_bias   [H P + 2 G N]        fp32       NULL = 0
 *   A           [H]                  fp32       normally < 0
 *   D, dt_bias  [H]                  fp32       NULL = 0
 *   lengths     [B]                  int32      tokens of each batch element,
 *                                               clamped to 0..L; NULL = L.
 *                                               Tokens past the end are not
 *                                               read, their y is zero, and the
 *                                               states are those after the last
 *                                               token inside
 *   h0          [B, H, P, N]         fp32       NULL = zero
 *   conv_state  [B, K-1, H P + 2 G N] in_dtype  NULL = zero
 *   y           [B, L, H, P]         out_dtype  (written)
 *   last_state  [B, H, P, N]         fp32       (written; NULL = skip); may not alias h0
 *   last_conv_state                  in_dtype   as conv_state (written; NULL =
 *                                               skip); may not alias it
 *
 * Outputs must not overlap inputs or each other (INVALID_ARG).
 * N in {16, 32, 64, 128}.  State, decays and sums are fp32, and so are products
 * in effect.  The sequence is worked on in chunks of 64 tokens (up to 32 tokens
 * one by one, fewer where the heads fill the GPU, 7 at least): a NaN or infinity in a token
 * reaches every y of its chunk and head, and what follows, and so does a Delta x
 * past 2^60.  Rows may overlap (a row stride of 0 repeats one).  Workspace as
 * for the other entry points.
 */
typedef struct {
    int64_t batch, seqlen, nheads, headdim, ngroups, dstate, width;
    int64_t xbc_row, xbc_batch, dt_row, dt_batch;
    int32_t in_dtype, out_dtype;
    void* workspace;
    size_t workspace_bytes;
} selscan_m2_conv_shape_t;

/* Bytes of workspace selscan_mamba2_conv_fwd needs (0 on a bad shape): for each
 * 64 tokens and group 114 KB (N = 128; 66 for 64, 42 for 32 and 16), 58 MB for 8
 * x 4096 with one group, and a state for each head of each segment that a
 * sequence is cut into (about one for each compute unit of the GPU in all, four
 * and more to a sequence where it has lengths); for short sequences that go token
 * by token B L (H P + 2 G N) fp32. */
size_t selscan_mamba2_conv_workspace_bytes(const selscan_m2_conv_shape_t* shape);

selscan_status_t selscan_mamba2_conv_fwd(const selscan_m2_conv_shape_t* shape, const void* xbc, const void* dt,
                                         const float* conv_weight, const float* conv_bias, const float* A,
                                         const float* D, const float* dt_bias, const int32_t* lengths,
                                         const float* h0, const void* conv_state, void* y, float* last_state,
                                         void* last_conv_state, void* stream);

/*
 * The mixer for one token: xbc [B, H P + 2 G N] (batch elements xbc_batch
 * apart), dt [B, H] (dt_batch apart), y [B, H, P]; state [B, H, P, N] fp32
 * (16-byte aligned) and conv_state [B, K-1, H P + 2 G N] are updated in place.
 * y, state and conv_state must not overlap xbc, dt or each other
 * (INVALID_ARG).  seqlen, xbc_row, dt_row and workspace are ignored.
 */
selscan_status_t selscan_mamba2_conv_step(const selscan_m2_conv_shape_t* shape, float* state, void* conv_state,
                                          const void* xbc, const void* dt, const float* conv_weight,
                                          const float* conv_bias, const float* A, const float* D,
                                          const float* dt_bias, void* y, void* stream);

/*
 * RMS norm with the residual sum or the mixer's gate in front of it, and an
 * output in 8 bits with scales.  For each row and group (groups of width = dim
 * / groups elements; 1 = the row):
 *
 *     s    = x + residual                    or, with a gate, x gate sigmoid(gate)
 *     rstd = 1 / sqrt(sum s^2 / width + eps)
 *     y    = s rstd weight
 *
 * and where out_dtype is SELSCAN_E4M3, for each block of scale_block elements
 * of a group (the last one may be shorter; 0: the group):
 *
 *     scale = max(max |y| / 448, 2^-126);  y8 = y / scale, rounded to nearest even
 *
 * of the fp32 y and the fp32 quotient: y's own roundings (a few of 2^-24) take a
 * y / scale next to a tie of two e4m3 values to either of them.  A NaN makes its
 * block's scale NaN.
 *   x            [rows, dim]  in_dtype
 *   residual     [rows, dim]  res_dtype   NULL = 0
 *   gate         [rows, dim]  in_dtype    rows gate_row elements apart; NULL =
 *                                         none; not with a residual (UNSUPPORTED)
 *   weight       [dim]        fp32        NULL = 1
 *   y            [rows, dim]  out_dtype   (written)
 *   residual_out [rows, dim]  res_dtype   s (written; NULL = skip; not with a
 *                                         gate)
 *   rstd         [rows, groups] fp32      (written; NULL = skip)
 *   scale        [rows, groups ceil(width / scale_block)]  fp32  (written with
 *                                         E4M3, where it is required)
 * y and residual_out may each be an input of the same type (y over x, s over
 * residual), rows where that has them; other overlaps are INVALID_ARG.
 * scale_block: 0, 32, 64, 128, 256 or 512.  Sums are fp32 over s before it is
 * rounded, fp64 over the pieces of groups longer than 8192.  rows, dim, groups >= 1, dim % groups == 0.  Workspace is used by
 * the gradients only.
 */
typedef struct {
    int64_t rows, dim, groups, gate_row, scale_block;
    int32_t in_dtype, res_dtype, out_dtype;
    float eps;
    void* workspace;
    size_t workspace_bytes;
} selscan_rms_shape_t;

selscan_status_t selscan_rms_norm_fwd(const selscan_rms_shape_t* shape, const void* x, const void* residual,
                                      const void* gate, const float* weight, void* y, void* residual_out, float* rstd,
                                      float* scale, void* stream);

/* Bytes of workspace selscan_rms_norm_bwd needs (0 on a bad shape). */
size_t selscan_rms_norm_bwd_workspace_bytes(const selscan_rms_shape_t* shape);

/*
 * Gradients of selscan_rms_norm_fwd:
 *
 *     w  = dy weight;  xhat = s rstd
 *     ds = rstd (w - xhat sum (w xhat) / width) + dresidual_out
 *     without a gate  dx = ds, dresidual = ds;    with one (s made again from
 *     x and gate)     dx = ds silu(gate), dgate = ds x silu'(gate)
 *     dweight = sum_r dy xhat
 *
 *   dy            [rows, dim]  out_dtype   (FP32 or BF16: the gradient of an
 *                                          8-bit y is that of its value)
 *   s             [rows, dim]  res_dtype   as written to residual_out (x itself
 *                                          without a residual); with a gate x,
 *                                          and res_dtype is in_dtype
 *   gate, weight               as in the forward call
 *   rstd          [rows, groups] fp32
 *   dresidual_out [rows, dim]  res_dtype   gradient of s from its other uses;
 *                                          NULL = 0; not with a gate
 *   dx            [rows, dim]  in_dtype    (written; NULL = skip)
 *   dresidual     [rows, dim]  res_dtype   (written; NULL = skip); not with a gate
 *   dgate         [rows, dim]  in_dtype    (written; NULL = skip); with a gate only
 *   dweight       [dim]        fp32        (written; NULL = skip)
 * dx, dresidual and dgate may each be an input of the same type, rows where that
 * has them (dresidual over dresidual_out); not dy, s or gate where dweight of
 * groups longer than 8192 is asked for.  Other overlaps are INVALID_ARG.
 * Sums over rows run in a fixed order: results are reproducible bit for bit.
 * Workspace as for the other entry points; none where dweight is NULL.
 */
selscan_status_t selscan_rms_norm_bwd(const selscan_rms_shape_t* shape, const void* dy, const void* s,
                                      const void* gate, const float* weight, const float* rstd,
                                      const void* dresidual_out, void* dx, void* dresidual, void* dgate,
                                      float* dweight, void* stream);

/* Message for the last failed call on this thread ("" after a success).
 * The string stays valid until the next call on the same thread. */
const char* selscan_last_error(void);

/* Library version string, e.g. "libselscan 0.1 gfx950". */
const char* selscan_version(void);

/* ---- Kernel timing (instrumentation for benchmarks) ---------------------
 * selscan_timing_enable(1) makes every later kernel launch of the entry
 * points, on any thread, record a HIP event before and after the kernel on
 * the call's own stream.  selscan_timing_collect waits for all events
 * recorded so far, writes at most max_entries per-kernel aggregates to `out`
 * (host memory owned by the caller; `name` points to a static string of the
 * library) in order of first launch, forgets those events and returns the
 * number of distinct kernels (which may exceed max_entries), or a negative
 * value on a bad argument (-1) or an event failure (-2).  Enabling adds two
 * event records per launch to the stream; leave it off for end-to-end
 * timing.  selscan_timing_enable returns SELSCAN_ERR_INVALID_ARG for values
 * other than 0 and 1. */
typedef struct {
    const char* name;   /* e.g. "m1_scan_output" */
    int64_t launches;
    double total_ms, min_ms, max_ms;
} selscan_kernel_time_t;

selscan_status_t selscan_timing_enable(int on);
int selscan_timing_collect(selscan_kernel_time_t* out, int max_entries);

#ifdef __cplusplus
}
#endif

#endif /* SELSCAN_H */
