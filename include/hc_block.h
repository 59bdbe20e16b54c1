/*
 * hc_block.h -- operators of a channels-last sequence block (included by hc.h).
 *
 * Rows of a map read as sequences (pixels) or of a camera stream (frames) pass
 * through blocks of norm, mixer and feed-forward product.  Beside the mixers of
 * hc_mixer.h:
 *   - layer norm over the channels of each row (forward, backward);
 *   - linear attention with a decay for each head (forward, backward, one
 *     token): a mixer whose state is a matrix a head, so that most of its work
 *     is products of matrices;
 *   - the gated feed-forward product (forward, backward).
 *
 * The conventions are those of hc_mixer.h: hc_rows tensors with any
 * non-negative strides for inputs, outputs whose rows overlap neither one
 * another nor an input, fp32 sums, statistics and states, lens as a length for
 * each sequence (rows at or past it are not used, whatever they hold; their
 * outputs and gradients are zeros), no allocation, calls asynchronous on
 * `stream`, errors before any launch, results that repeat bit for bit.
 */
#ifndef HC_BLOCK_H
#define HC_BLOCK_H

#ifndef HC_H
#include "hc.h"
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* ---- layer norm ----------------------------------------------------------
 * x is [B][L][C].  For each row over its C values: mean, biased variance,
 * rstd = 1 / sqrt(var + eps), xhat = (x - mean) * rstd, y = gamma * xhat + beta.
 * Invalid: B, C < 1, L < 0, eps < 0 (HC_ERR_INVALID_ARG).  C <= 2^20 and
 * B * L < 2^31 (HC_ERR_UNSUPPORTED beyond). */
typedef struct {
    int B, L, C;
    float eps;
    int dtype; /* hc_dtype */
} hc_layernorm_desc;

/* Forward.  mean and rstd ([B][L], may be NULL) keep the statistics for the
 * backward pass (zeros at rows past a sequence's end). */
hc_status hc_layernorm_fwd(const hc_layernorm_desc* d, const hc_rows* x, const float* gamma, const float* beta,
                           const hc_rows* y, float* mean, float* rstd, const int* lens, void* stream);

/* Workspace bytes of hc_layernorm_bwd. */
hc_status hc_layernorm_workspace_size(const hc_layernorm_desc* d, size_t* bytes);

/* Backward: with q = gamma * gy, gx = rstd * (q - mean(q) - xhat * mean(q * xhat)),
 * the means over the row's channels; ggamma = sum gy * xhat and gbeta = sum gy
 * over the rows (either may be NULL; zeros if there is no row). */
hc_status hc_layernorm_bwd(const hc_layernorm_desc* d, const hc_rows* x, const float* gamma, const float* mean,
                           const float* rstd, const hc_rows* gy, const hc_rows* gx, float* ggamma, float* gbeta,
                           const int* lens, void* ws, size_t ws_bytes, void* stream);

/* ---- linear attention with a decay for each head --------------------------
 * q and k are [B][L][H * Dk], v and y [B][L][H * Dv]: heads adjacent in a row.
 * With lambda = exp(log_decay[h]) ([H], at most 0; NULL: no decay), for each
 * head from h0 ([B][H][Dk][Dv] fp32, NULL: zeros):
 *   S_t = lambda * S_{t-1} + k_t v_t^T,     y_t = scale * q_t S_t.
 * hT (may be NULL): the state behind the sequence's last row.  A log decay of
 * minus infinity forgets everything but the row itself; one above 0 is not
 * checked.  The decay is a constant of the head: it has no gradient.
 * 1 <= Dk, Dv <= 128, L < 2^31 - 256, H * Dk and H * Dv <= 2^20, B * H < 2^31 /
 * 3 (HC_ERR_UNSUPPORTED beyond); sizes < 1 (L < 0) and a scale that is not
 * finite are HC_ERR_INVALID_ARG.
 * Arithmetic: bf16 rows go through the tensor cores where Dk and Dv are multiples
 * of 8, addresses and strides multiples of 16 bytes (strides not 0) and L is more
 * than 32 (8 where Dk or Dv is above 32, 0 where one is above 64): scores, and the
 * state as it is read, are rounded once to bf16 there; the state itself is fp32.
 * All others are multiplied in fp32.
 * Rows are taken in chunks of up to 128: a value that is not finite may spoil its
 * whole chunk, not only the rows behind it. */
typedef struct {
    int B, L, H, Dk, Dv;
    float scale;
    int dtype; /* hc_dtype */
} hc_linear_attn_desc;

/* Workspace bytes of hc_linear_attn_fwd (pass 0) or of both passes (pass 1). */
hc_status hc_linear_attn_workspace_size(const hc_linear_attn_desc* d, int pass, size_t* bytes);

hc_status hc_linear_attn_fwd(const hc_linear_attn_desc* d, const hc_rows* q, const hc_rows* k, const hc_rows* v,
                             const float* log_decay, const hc_rows* y, const float* h0, float* hT, const int* lens,
                             void* ws, size_t ws_bytes, void* stream);

/* Backward, from the inputs alone (the states are computed again).  With the
 * state's gradient G_t = scale * q_t gy_t^T + lambda * G_{t+1} (behind the last
 * row: lambda * G is ghT, [B][H][Dk][Dv], NULL: zeros):
 *   gq_t = scale * S_t gy_t,  gk_t = G_t v_t,  gv_t = G_t^T k_t,
 *   gh0 = lambda * G_0 (may be NULL; ghT for a sequence without rows). */
hc_status hc_linear_attn_bwd(const hc_linear_attn_desc* d, const hc_rows* q, const hc_rows* k, const hc_rows* v,
                             const float* log_decay, const float* h0, const hc_rows* gy, const float* ghT,
                             const hc_rows* gq, const hc_rows* gk, const hc_rows* gv, float* gh0, const int* lens,
                             void* ws, size_t ws_bytes, void* stream);

/* One token of every sequence: q, k are [B][H * Dk], v, y [B][H * Dv] (row
 * strides and the desc's L are not used); state is read and updated in place. */
hc_status hc_linear_attn_step(const hc_linear_attn_desc* d, const hc_rows* q, const hc_rows* k, const hc_rows* v,
                              const float* log_decay, float* state, const hc_rows* y, void* stream);

/* ---- gated feed-forward product --------------------------------------------
 * x and y are [M][C] (batch strides are not used), w_in is [C][2 F] (F gate
 * columns, then F value columns) and w_out [F][C], contiguous and 16-byte
 * aligned, all of the desc's type, HC_DTYPE_BF16 or HC_DTYPE_F16:
 *   a = x w_in[:, :F],  u = x w_in[:, F:],  h = act(a) * u,  y = h w_out,
 * act an hc_pw_act.  Products are summed in fp32; h is rounded once to the
 * desc's type, y once.  In fp16 a value of h, or of ga and gu below, beyond 65504
 * is infinite, and its row of y or gx and the gradients of the weights that it
 * enters are infinite or NaN; one below 2^-25 is zero (bf16 has fp32's range).
 * C and F are multiples of 8 up to 2^16, rows start on 16-byte boundaries
 * (address, row stride, which is not 0), M < 2^31 - 256, M * C and M * F at most
 * 2^38: HC_ERR_UNSUPPORTED otherwise, and for fp32.  M = 0 is a valid call. */
typedef struct {
    int M, C, F;
    int act;   /* hc_pw_act */
    int dtype; /* hc_dtype */
} hc_gated_ffn_desc;

/* Workspace bytes of hc_gated_ffn_fwd (pass 0) or of both passes (pass 1). */
hc_status hc_gated_ffn_workspace_size(const hc_gated_ffn_desc* d, int pass, size_t* bytes);

hc_status hc_gated_ffn_fwd(const hc_gated_ffn_desc* d, const hc_rows* x, const void* w_in, const void* w_out,
                           const hc_rows* y, void* ws, size_t ws_bytes, void* stream);

/* Backward, from the inputs alone (a and u are computed again).  With
 * gh = gy w_out^T, ga = gh * u * act'(a), gu = gh * act(a) (each rounded once):
 *   gx = ga w_in[:, :F]^T + gu w_in[:, F:]^T,
 *   gw_in = x^T [ga | gu] ([C][2 F]),  gw_out = h^T gy ([F][C]),
 * both contiguous and of the desc's type; each of the three may be NULL.  No
 * gradient of the weights overlaps another gradient or an input, and neither gx
 * nor, in the forward pass, y the weights (HC_ERR_INVALID_ARG). */
hc_status hc_gated_ffn_bwd(const hc_gated_ffn_desc* d, const hc_rows* x, const void* w_in, const void* w_out,
                           const hc_rows* gy, const hc_rows* gx, void* gw_in, void* gw_out, void* ws, size_t ws_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HC_BLOCK_H */
