/*
 * dn_window_ops.h -- C ABI of attention over a sliding window with sinks: the
 * layers that stand between those of the gated delta rule in a stack of both.
 *
 * With w = window and s = sinks, token t of a sequence sees the tokens
 *
 *     V(t) = { j : t - w < j <= t }  and  { j : j < s, j <= t },
 *
 * itself among them, so that no token sees nothing.  For query head h and
 * key head h / (Nq / Nk):
 *
 *     p_tj = e^{scale q_t . k_j - lse_t},  lse_t = log sum_{j in V(t)} e^{scale q_t . k_j}
 *     o_t  = sum_{j in V(t)} p_tj v_j
 *
 * A window of T or more is plain causal attention.
 *
 * The conventions are those of dn_layer_ops.h: device memory of the current
 * device, contiguous, 16-byte aligned; asynchronous and ordered on `stream`;
 * sequences and their offsets; outputs overlap no input and no other output
 * except where an entry point says so; argument errors are found on the host.
 * Scores, the softmax's maxima and sums, and all accumulators are fp32.  With
 * bf16 tensors the products run on the tensor cores: the weights p (and in the
 * backward ds = p (dp - D)) are rounded to bf16 for them.  With fp32 tensors
 * every product is fp32.  Results do not depend on the order in which blocks run.
 *
 * What a masked key or its value holds (NaN and infinities too) reaches no
 * output.  A row whose own operands are not finite comes out as the formulas
 * say; it costs a second, slower pass over its tile, as does one of bf16 whose
 * scores rise by 85 and more from one tile of 128 keys to a later one.
 *
 * Limits beside those of the entry points (DN_ERR_UNSUPPORTED): B T <= 2^31 - 256,
 * T <= 2^30.
 */
#ifndef DN_WINDOW_OPS_H
#define DN_WINDOW_OPS_H

#include "dn_layer_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * dn_window_attn_fwd
 *   q       [B, T, Nq, d]  dtype
 *   k, v    [B, T, Nk, d]  dtype    Nq % Nk == 0
 *   window  w >= 1;  sinks  0 <= s <= 128 (more: DN_ERR_UNSUPPORTED)
 *   scale   <= 0 selects 1 / sqrt(d)
 *   o       [B, T, Nq, d]  dtype
 *   lse     [B, T, Nq]     float32  (required: the backward reads it)
 * d is 64 or 128 (else DN_ERR_UNSUPPORTED).
 */
dn_status dn_window_attn_fwd(const void *q, const void *k, const void *v, const int64_t *cu_seqlens, int n_seqs, int B,
                             int T, int Nq, int Nk, int d, int window, int sinks, dn_dtype dtype, float scale, void *o,
                             float *lse, dn_stream_t stream);

/*
 * dn_window_attn_bwd -- gradients of q, k and v for the loss sum(d_o . o); o
 * and lse are what dn_window_attn_fwd gave for the same inputs.
 *   d_o            [B, T, Nq, d]  dtype
 *   d_q            [B, T, Nq, d]  dtype
 *   d_k, d_v       [B, T, Nk, d]  dtype   summed over the group's query heads
 * workspace: dn_window_attn_bwd_workspace_bytes() bytes (packed: 1 with
 * cu_seqlens, else 0).
 */
dn_status dn_window_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                             const int64_t *cu_seqlens, int n_seqs, int B, int T, int Nq, int Nk, int d, int window,
                             int sinks, dn_dtype dtype, float scale, const void *d_o, void *d_q, void *d_k, void *d_v,
                             void *workspace, size_t workspace_bytes, dn_stream_t stream);

size_t dn_window_attn_bwd_workspace_bytes(int packed, int n_seqs, int B, int T, int Nq, int Nk, int d, int window,
                                          int sinks, dn_dtype dtype);

/*
 * The ring cache of a sequence's keys and values: for every key head `sinks`
 * slots and then `ring` slots.  The token at position p (from 0) has slot p
 * where p < sinks, else sinks + (p - sinks) % ring.  Slots that no token has
 * been written to are not read.
 *
 * dn_window_cache_fill -- puts the tokens of k and v into the caches; of those
 * that share a slot the last one stays.
 *   k, v              [B, T, Nk, d]  dtype  (cu_seqlens as above)
 *   lengths           [n_seqs]       int64  tokens that each sequence had
 *                                           before these; NULL: none
 *   k_cache, v_cache  [n_seqs, Nk, sinks + ring, d]  dtype
 * d is 64 or 128; ring >= 1, sinks + ring <= 2^30; Nk <= 65536.  A length that is negative, or
 * that 64 bits do not hold with the tokens added, makes dn_check return
 * DN_ERR_DEVICE_ARG; nothing is written for that sequence.
 */
dn_status dn_window_cache_fill(const void *k, const void *v, const int64_t *cu_seqlens, int n_seqs, int B, int T,
                               int Nk, int d, int sinks, int ring, dn_dtype dtype, const int64_t *lengths,
                               void *k_cache, void *v_cache, dn_stream_t stream);

/*
 * dn_window_attn_step -- one new token of every sequence: its key and value
 * go into the caches, and its queries see what the formula above lets the
 * token at position lengths[n] see.
 *   q        [n_seqs, Nq, d], k, v [n_seqs, Nk, d], o [n_seqs, Nq, d]  dtype
 *   lengths  [n_seqs] int64  tokens in the cache before the call (not changed)
 * window <= ring, sinks + ring <= 2^30; n_seqs Nq <= 2^27 - 16.  scale as above.  A negative length makes dn_check return
 * DN_ERR_DEVICE_ARG and leaves that sequence's outputs unspecified.
 */
dn_status dn_window_attn_step(const void *q, const void *k, const void *v, int n_seqs, int Nq, int Nk, int d, int window,
                              int sinks, int ring, dn_dtype dtype, float scale, const int64_t *lengths, void *k_cache,
                              void *v_cache, void *o, dn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DN_WINDOW_OPS_H */
