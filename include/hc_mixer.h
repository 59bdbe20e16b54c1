/*
 * hc_mixer.h -- channels-last sequence-mixer operators (included by hc.h).
 *
 * After the convolution stages a feature map is read as sequences of pixels
 * (or a camera stream as a sequence of frames).  Three operators mix along
 * such a sequence at a cost linear in its length:
 *   - group norm with an activation, channels last (forward, backward);
 *   - a short causal depthwise convolution (forward, backward, one token);
 *   - a selective state-space scan (forward, backward, one token).
 * A sequence split over W shards hands the convolution's last K - 1 rows and
 * the scan's state from one block to the next: they are the one-sided halo of
 * this path, and both are inputs and outputs of the calls.
 *
 * Conventions, beyond those of hc.h (the caller owns every buffer, calls are
 * asynchronous on `stream`, errors come before any launch, results repeat bit
 * for bit):
 *   - A channels-last tensor [batch][row][channel] is passed as an hc_rows:
 *     address, element strides of batch and row, element type.  Channels are
 *     adjacent.  Inputs may have any non-negative strides (slices of wider
 *     rows, broadcasts); an output's rows must not overlap one another, nor
 *     any input's.  Addresses need the alignment of their element type;
 *     16-byte aligned addresses and strides take the wide loads.
 *   - Elements are fp32, bf16 or fp16 (one type per call, that of the desc).
 *     Sums, statistics, states and exponentials are fp32; each output element
 *     is rounded once, when it is stored.  Parameters (gamma, beta, weights,
 *     bias, A, D, dt_bias), their gradients, the norm's statistics and the
 *     scan's states are fp32 arrays, contiguous and 16-byte aligned.
 *   - lens (NULL: every sequence has all L rows) gives each sequence's length
 *     in device memory, taken as within 0 .. L.  Rows at or past it are not
 *     used, whatever they hold; their outputs and gradients are zeros.
 *   - L = 0 is a valid call: states pass through, nothing else is written
 *     (parameter gradients become zero).
 *   - Sizes past these limits are HC_ERR_UNSUPPORTED.  Norm: N <= 65535,
 *     C <= 2^20, N * groups < 2^30.  Convolution: 2 <= K <= 8, D <= 2^20,
 *     B * (L / 4 + 1) < 2^31, L < 2^31 - 64.  Scan: d_state <= 64, D <= 2^20,
 *     B * D < 2^31, L < 2^31 - 64.
 */
#ifndef HC_MIXER_H
#define HC_MIXER_H

#ifndef HC_H
#include "hc.h"
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { HC_DTYPE_F32 = 0, HC_DTYPE_BF16 = 1, HC_DTYPE_F16 = 2 } hc_dtype;
/* Activations of the norm and the convolution: x, x / (1 + exp(-x)) and
 * x * (1 + erf(x / sqrt 2)) / 2 (no further from it than hc_gelu_fwd, and with
 * its negative tail to a relative 1e-5). */
typedef enum { HC_PW_NONE = 0, HC_PW_SILU = 1, HC_PW_GELU = 2 } hc_pw_act;

typedef struct {
    void* p;              /* NULL: the tensor is absent (where that is allowed) */
    long long batch, row; /* element strides */
    long long dtype;      /* an hc_dtype */
} hc_rows;

/* ---- group norm with an activation --------------------------------------
 * x is [N][P][C] (P pixels an image); channels split into `groups` equal runs.
 * For image n and group g over its P * C / groups values: mean, biased
 * variance, rstd = 1 / sqrt(var + eps), xhat = (x - mean) * rstd and
 * y = act(gamma[c] * xhat + beta[c]).
 * Invalid: sizes < 1, C % groups != 0, eps < 0 (HC_ERR_INVALID_ARG). */
typedef struct {
    int N, P, C, groups;
    float eps;
    int act;   /* hc_pw_act */
    int dtype; /* hc_dtype  */
} hc_groupnorm_desc;

/* Workspace bytes of hc_groupnorm_fwd (pass 0) or of both passes (pass 1). */
hc_status hc_groupnorm_workspace_size(const hc_groupnorm_desc* d, int pass, size_t* bytes);

/* Forward.  mean and rstd ([N][groups], may be NULL) keep the statistics for
 * the backward pass. */
hc_status hc_groupnorm_fwd(const hc_groupnorm_desc* d, const hc_rows* x, const float* gamma, const float* beta,
                           const hc_rows* y, float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream);

/* Backward: with g = gy * act'(gamma * xhat + beta), ggamma[c] = sum g * xhat
 * and gbeta[c] = sum g over n and pixels (either may be NULL), and with
 * q = gamma[c] * g, gx = rstd * (q - mean(q) - xhat * mean(q * xhat)), the
 * means over the group's values. */
hc_status hc_groupnorm_bwd(const hc_groupnorm_desc* d, const hc_rows* x, const float* gamma, const float* beta,
                           const float* mean, const float* rstd, const hc_rows* gy, const hc_rows* gx, float* ggamma,
                           float* gbeta, void* ws, size_t ws_bytes, void* stream);

/* ---- short causal depthwise convolution ----------------------------------
 * x is [B][L][D]; w is [D][K], 2 <= K <= 8 (HC_ERR_UNSUPPORTED beyond), bias
 * [D] (may be NULL).  With rows before the first taken from state_in
 * ([B][K-1][D] contiguous, elements of the desc's type; NULL: zeros):
 *   pre_t = bias + sum_k w[k] * x_{t - (K-1) + k},  y_t = act(pre_t),
 * act HC_PW_NONE or HC_PW_SILU.  state_out (may be NULL): the last K - 1 rows
 * up to the sequence's end, those of state_in among them if it is shorter.
 * state_out may be state_in's own buffer only in hc_causal_conv_step. */
typedef struct {
    int B, L, D, K;
    int act;   /* HC_PW_NONE, HC_PW_SILU */
    int dtype; /* hc_dtype */
} hc_causal_conv_desc;

hc_status hc_causal_conv_fwd(const hc_causal_conv_desc* d, const hc_rows* x, const float* w, const float* bias,
                             const hc_rows* y, const void* state_in, void* state_out, const int* lens, void* stream);

/* Workspace bytes of hc_causal_conv_bwd. */
hc_status hc_causal_conv_workspace_size(const hc_causal_conv_desc* d, size_t* bytes);

/* Backward: with g_t = gy_t * act'(pre_t), gx_t = sum_k w[k] * g_{t+K-1-k},
 * gw[d][k] = sum over b, t of g_t * x_{t-(K-1)+k}, gb[d] = sum g_t.
 * gstate_out (may be NULL): the gradient of state_out, which joins that of the
 * rows it holds.  gstate_in (may be NULL): the gradient of state_in.  Both are
 * [B][K-1][D] in the desc's type.  gstate_in may be neither gstate_out's nor
 * state_in's own buffer: other blocks still read those.  gx, gw, gb may each be
 * NULL. */
hc_status hc_causal_conv_bwd(const hc_causal_conv_desc* d, const hc_rows* x, const float* w, const float* bias,
                             const hc_rows* gy, const hc_rows* gx, float* gw, float* gb, const void* state_in,
                             const void* gstate_out, void* gstate_in, const int* lens, void* ws, size_t ws_bytes,
                             void* stream);

/* One token of every sequence: x and y are [B][D] (the row stride is not
 * used; the desc's L is not used); state [B][K-1][D] is read and then moved on
 * by one row in place. */
hc_status hc_causal_conv_step(const hc_causal_conv_desc* d, const hc_rows* x, const float* w, const float* bias,
                              void* state, const hc_rows* y, void* stream);

/* ---- selective state-space scan -------------------------------------------
 * u, dt, z, y are [B][L][D]; Bm and Cm are [B][L][groups * d_state], group g
 * serving channels g * D/groups .. (g+1) * D/groups - 1; A is [D][d_state].
 * For channel d and state n, from h0 ([B][D][d_state], NULL: zeros):
 *   delta_t = softplus(dt_t + dt_bias[d])   (or dt_t + dt_bias[d])
 *   h_t[n]  = exp(delta_t * A[d][n]) * h_{t-1}[n] + delta_t * u_t * Bm_t[n]
 *   y_t     = (sum_n Cm_t[n] * h_t[n] + D[d] * u_t) * silu(z_t)
 * z, D and dt_bias may be absent (no gate, 0, 0).  hT (may be NULL) is the
 * state after the sequence's last row.  1 <= d_state <= 64
 * (HC_ERR_UNSUPPORTED beyond); D % groups == 0.  delta_t * A is expected to be
 * at most 0 (a state that does not grow), but is not checked. */
typedef struct {
    int B, L, D, groups, d_state;
    int softplus; /* 0 or 1 */
    int dtype;    /* hc_dtype */
} hc_selective_scan_desc;

typedef struct {
    hc_rows u, dt, Bm, Cm, z;
    const float *A, *D, *dt_bias;
} hc_scan_in;

typedef struct {
    hc_rows gu, gdt, gB, gC, gz; /* laid out as u, dt, Bm, Cm, z; gz absent without z */
    float *gA, *gD, *gdt_bias;   /* gD, gdt_bias may be NULL */
    float* gh0;                  /* may be NULL */
} hc_scan_grad;

/* Workspace bytes of hc_selective_scan_fwd (pass 0) or of both passes
 * (pass 1), and the bytes of the states that the forward pass saves for the
 * backward one. */
hc_status hc_selective_scan_workspace_size(const hc_selective_scan_desc* d, int pass, size_t* bytes);
hc_status hc_selective_scan_saved_size(const hc_selective_scan_desc* d, size_t* bytes);

/* Forward.  saved (NULL when there is no backward pass): 16-byte aligned. */
hc_status hc_selective_scan_fwd(const hc_selective_scan_desc* d, const hc_scan_in* in, const float* h0,
                                const int* lens, const hc_rows* y, float* hT, void* saved, void* ws, size_t ws_bytes,
                                void* stream);

/* Backward of a forward pass on the same inputs with `saved`: the gradients of
 * u, dt, Bm, Cm, z, A, D, dt_bias and h0.  With q_t = gy_t * silu(z_t) and the
 * state's gradient G_t = q_t Cm_t + exp(delta_{t+1} A) G_{t+1} (after the last
 * row: ghT, [B][D][d_state], NULL: zeros), E_t = G_t exp(delta_t A) h_{t-1}:
 *   gBm = sum_d delta u G     gCm = sum_d q h       gA = sum_{b,t} delta E
 *   gu = delta (G . Bm) + D q                       gD = sum_{b,t} q u
 *   gdelta = u (G . Bm) + E . A                     gh0 = exp(delta_0 A) G_0
 *   gdt = gdelta * softplus'(dt + dt_bias), gdt_bias its sum over b and t,
 *   gz = gy * (C . h + D u) * silu'(z);
 * gBm and gCm sum over the channels of a group. */
hc_status hc_selective_scan_bwd(const hc_selective_scan_desc* d, const hc_scan_in* in, const float* h0,
                                const int* lens, const void* saved, const hc_rows* gy, const float* ghT,
                                const hc_scan_grad* g, void* ws, size_t ws_bytes, void* stream);

/* One token of every sequence: u, dt, z, y are [B][D], Bm and Cm
 * [B][groups * d_state] (row strides and the desc's L are not used); state
 * [B][D][d_state] is read and updated in place. */
hc_status hc_selective_scan_step(const hc_selective_scan_desc* d, const hc_scan_in* in, float* state, const hc_rows* y,
                                 void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HC_MIXER_H */
