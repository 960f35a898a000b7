/*
 * dn_layer_ops.h -- C ABI of the operators around the gated delta rule in a
 * layer: the short causal convolution that q, k and v pass before the
 * recurrence, the selective state space scan (a recurrence with a decay of
 * its own for every channel and state), and layer norm with its
 * root-mean-square form and its output gate.  Each has a forward and a
 * backward entry point; the single-token form of the convolution and of the
 * scan is the forward with T = 1, h0 in and ht out, as for dn_recurrent_fwd.
 *
 * The conventions are those of dn_chunk_fwd.h:
 *   - all tensors are device memory of the current device, owned by the
 *     caller, row-major and contiguous, 16-byte aligned (a row may be of any
 *     length: only the first element is aligned); the library keeps no
 *     reference and allocates nothing; workspaces are the caller's, 16-byte
 *     aligned, and not touched by anyone else until the stream has passed the
 *     call; their contents on entry do not matter;
 *   - calls are asynchronous and ordered on `stream`, and can be captured
 *     into a CUDA graph;
 *   - outputs overlap no input and no other output, except where an entry
 *     point says so;
 *   - argument errors are found on the host before anything is launched.
 *
 * Sequences.  With cu_seqlens NULL there are n_seqs = B sequences of length
 * T.  Otherwise B == 1 and sequence n is the tokens [cu[n], cu[n+1]) of T;
 * cu must start at 0, not decrease and end at most at T.  It is read on the
 * device: a malformed one makes dn_check return DN_ERR_DEVICE_ARG and leaves
 * the outputs unspecified; nothing outside the tensors is touched.  Rows of
 * tokens behind the last sequence are not written.  A sequence may be empty:
 * its final state is its initial one.  T is at most 2^30 (larger:
 * DN_ERR_UNSUPPORTED).
 *
 * Every sum, state and statistic is held in fp32.  Outputs of type `dtype`
 * are rounded to it once (to nearest even).  Results do not depend on the
 * order in which blocks run: the same call gives the same bits.  Exponentials
 * and quotients are the hardware's approximate ones, for fp32 tensors too:
 * fp32 outputs are up to about 3 times as far from exact ones as those of the
 * formulas evaluated with the standard fp32 functions.
 */
#ifndef DN_LAYER_OPS_H
#define DN_LAYER_OPS_H

#include "dn_chunk_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Option bit of dn_causal_conv_*: y = u / (1 + e^-u) of the convolution u. */
#define DN_CONV_SILU 1u
/* Option bit of dn_selective_scan_*: delta = log(1 + e^(dt + dt_bias)). */
#define DN_SCAN_SOFTPLUS 1u
/* Option bit of dn_layer_norm_*: no mean is taken (root mean square norm). */
#define DN_NORM_RMS 1u

/*
 * dn_causal_conv_fwd -- depthwise causal convolution over the last W tokens.
 *
 *     u_t[d] = bias[d] + sum_{j < W} weight[d, j] x_{t - (W-1) + j}[d]
 *     y_t    = u_t, or silu(u_t) with DN_CONV_SILU
 *
 * where a token before the sequence's first is a row of h0 (the last row is
 * the nearest one), or zero.
 *   x       [B, T, D]       dtype
 *   weight  [D, W]          float32   W = 2, 3 or 4, the last tap the token's own
 *   bias    [D]             float32   or NULL: zero
 *   h0      [n_seqs, W-1, D] dtype    inputs before the sequence; NULL: zero
 *   y       [B, T, D]       dtype
 *   ht      [n_seqs, W-1, D] dtype    the last W-1 inputs, those of h0 among
 *                                     them where the sequence is shorter;
 *                                     NULL: not written.  May be h0 itself.
 * D >= 1.  Another W is DN_ERR_UNSUPPORTED.
 */
dn_status dn_causal_conv_fwd(const void *x, const float *weight, const float *bias, const void *h0,
                             const int64_t *cu_seqlens, int n_seqs, int B, int T, int D, int W,
                             dn_dtype dtype, unsigned flags, void *y, void *ht, dn_stream_t stream);

/*
 * dn_causal_conv_bwd -- gradients of dn_causal_conv_fwd's inputs for the loss
 * sum(d_y . y) + sum(d_ht . ht).
 *   d_y      [B, T, D]        dy_dtype  dtype, or DN_F32 (as dn_chunk_bwd
 *                                       writes the gradients of q, k and v)
 *   d_ht     [n_seqs, W-1, D] dtype     NULL: zero
 *   d_x      [B, T, D]        dtype
 *   d_weight [D, W]           float32
 *   d_bias   [D]              float32   NULL: not computed; with bias NULL it
 *                                       is the gradient at bias = 0
 *   d_h0     [n_seqs, W-1, D] dtype     NULL: not computed; with h0 NULL it
 *                                       is the gradient at h0 = 0
 * d_weight and d_bias are written whatever the lengths (zero without tokens).
 * workspace: dn_causal_conv_bwd_workspace_bytes() bytes.
 */
dn_status dn_causal_conv_bwd(const void *x, const float *weight, const float *bias, const void *h0,
                             const int64_t *cu_seqlens, int n_seqs, int B, int T, int D, int W,
                             dn_dtype dtype, unsigned flags, const void *d_y, dn_dtype dy_dtype,
                             const void *d_ht, void *d_x, float *d_weight, float *d_bias, void *d_h0,
                             void *workspace, size_t workspace_bytes, dn_stream_t stream);

/* Bytes of workspace dn_causal_conv_bwd needs (0 for sizes it rejects). */
size_t dn_causal_conv_bwd_workspace_bytes(int n_seqs, int B, int T, int D, int W, dn_dtype dtype);

/*
 * dn_selective_scan_fwd -- the selective state space recurrence.  For channel
 * d of group g = d / (D / G) and state n < N, from h = h0 (or 0):
 *
 *     delta   = dt_t[d] + dt_bias[d], through log(1 + e^.) with DN_SCAN_SOFTPLUS
 *     h[n]    = e^{delta A[d, n]} h[n] + delta Bm_t[g, n] x_t[d]
 *     y_t[d]  = (sum_n Cm_t[g, n] h[n] + Dskip[d] x_t[d]) silu(z_t[d])
 *
 *   x, dt    [B, T, D]       dtype
 *   A        [D, N]          float32
 *   Bm, Cm   [B, T, G, N]    dtype
 *   Dskip    [D]             float32   or NULL: no such term
 *   z        [B, T, D]       dtype     or NULL: no factor silu(z)
 *   dt_bias  [D]             float32   or NULL: zero
 *   h0, ht   [n_seqs, D, N]  float32   NULL: zero / not written.  ht may be h0.
 *   y        [B, T, D]       dtype
 * D % G == 0; N is 16, 32, 64 or 128 (else DN_ERR_UNSUPPORTED).
 * workspace: dn_selective_scan_fwd_workspace_bytes() bytes (may be NULL when
 * that is 0, as it is for single tokens).
 */
dn_status dn_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *Bm,
                                const void *Cm, const float *Dskip, const void *z,
                                const float *dt_bias, const float *h0, const int64_t *cu_seqlens,
                                int n_seqs, int B, int T, int D, int G, int N, dn_dtype dtype,
                                unsigned flags, void *y, float *ht, void *workspace,
                                size_t workspace_bytes, dn_stream_t stream);

size_t dn_selective_scan_fwd_workspace_bytes(int n_seqs, int B, int T, int D, int G, int N,
                                             dn_dtype dtype);

/*
 * dn_selective_scan_bwd -- gradients of dn_selective_scan_fwd's inputs for the
 * loss sum(d_y . y) + sum(d_ht . ht).
 *   d_y             [B, T, D]      dtype
 *   d_ht            [n_seqs, D, N] float32  NULL: zero
 *   d_x, d_dt, d_z  [B, T, D]      dtype    d_z is required exactly when z is given
 *   d_A             [D, N]         float32
 *   d_Bm, d_Cm      [B, T, G, N]   dtype    summed over the group's channels
 *   d_Dskip, d_dt_bias [D]         float32  NULL: not computed
 *   d_h0            [n_seqs, D, N] float32  NULL: not computed.  May be d_ht.
 * d_A, d_Dskip and d_dt_bias are written whatever the lengths.
 * workspace: dn_selective_scan_bwd_workspace_bytes() bytes.
 */
dn_status dn_selective_scan_bwd(const void *x, const void *dt, const float *A, const void *Bm,
                                const void *Cm, const float *Dskip, const void *z,
                                const float *dt_bias, const float *h0, const int64_t *cu_seqlens,
                                int n_seqs, int B, int T, int D, int G, int N, dn_dtype dtype,
                                unsigned flags, const void *d_y, const float *d_ht, void *d_x,
                                void *d_dt, float *d_A, void *d_Bm, void *d_Cm, float *d_Dskip,
                                void *d_z, float *d_dt_bias, float *d_h0, void *workspace,
                                size_t workspace_bytes, dn_stream_t stream);

size_t dn_selective_scan_bwd_workspace_bytes(int n_seqs, int B, int T, int D, int G, int N,
                                             dn_dtype dtype);

/*
 * dn_layer_norm_fwd -- norm of every row of length D, then weight, bias, gate.
 *
 *     m = mean(x) (0 with DN_NORM_RMS),  r = 1 / sqrt(mean((x - m)^2) + eps)
 *     y = ((x - m) r weight + bias) silu(z)
 *
 *   x, z, y  [rows, D]  dtype    z NULL: no factor silu(z).  y may be x or z.
 *   weight   [D]        float32  NULL: one
 *   bias     [D]        float32  NULL: zero
 * The squares are taken in fp32: those of values beyond 1e19 overflow (y is 0),
 * those of values below 1e-23 are 0 (with eps = 0 and no larger value in the
 * row, y is not finite).
 * 1 <= D <= 16384 (larger: DN_ERR_UNSUPPORTED); rows >= 0; eps >= 0, finite.
 */
dn_status dn_layer_norm_fwd(const void *x, const float *weight, const float *bias, const void *z,
                            int64_t rows, int D, dn_dtype dtype, float eps, unsigned flags, void *y,
                            dn_stream_t stream);

/*
 * dn_layer_norm_bwd -- gradients of dn_layer_norm_fwd's inputs for the loss
 * sum(d_y . y); the row statistics are computed again from x.
 *   d_y, d_x, d_z  [rows, D]  dtype    d_z is required exactly when z is given
 *   d_weight       [D]        float32  NULL: not computed; with weight NULL it
 *                                      is the gradient at weight = 1
 *   d_bias         [D]        float32  NULL: not computed; with bias NULL it
 *                                      is the gradient at bias = 0
 * d_weight and d_bias are sums over all rows (zero for rows = 0).  d_x may be
 * d_y or x, d_z may be z.
 * workspace: dn_layer_norm_bwd_workspace_bytes() bytes (for either of
 * d_weight and d_bias; else it may be NULL).
 */
dn_status dn_layer_norm_bwd(const void *x, const float *weight, const float *bias, const void *z,
                            int64_t rows, int D, dn_dtype dtype, float eps, unsigned flags,
                            const void *d_y, void *d_x, float *d_weight, float *d_bias, void *d_z,
                            void *workspace, size_t workspace_bytes, dn_stream_t stream);

size_t dn_layer_norm_bwd_workspace_bytes(int64_t rows, int D, dn_dtype dtype);

#ifdef __cplusplus
}
#endif

#endif /* DN_LAYER_OPS_H */
