/*
 * carve_mixers.h -- C ABI of two further token mixers of libcarve.so (B200, sm_100a), beside the
 * CARVE recurrence of carve.h: the scalar-gated delta rule and sliding-window attention with
 * sink tokens, the two other layers of a hybrid recurrent / local-attention stack.  The
 * conventions are those of carve.h: stream-ordered on the caller's stream, no allocation, no
 * synchronisation, DEVICE pointers owned by the caller, arguments validated on the host before any
 * launch, a rejected call launches nothing and returns a non-zero carve_status.  Tensors with a
 * channel axis, states, caches and buffers are 16-byte aligned; gates, offsets, positions, lse and
 * the decay's parameters need their element's alignment only.  No entry point keeps state between calls, so concurrent calls on different
 * streams are safe when their outputs, saved buffers and workspaces are disjoint (this includes
 * captured graphs: two graphs that may run at once need two workspaces).
 *
 * Packed sequences: a non-NULL cu_seqlens (DEVICE int32 [B+1], non-decreasing) packs B sequences
 * along the token axis without padding: sequence n owns rows [cu[n], cu[n+1]) of [total_tokens,
 * heads, channels] tensors, and T is ignored.  Lengths from 0 are allowed; rows that belong to
 * no sequence reach no result and are not written.  The offsets live on the device: a sequence whose
 * rows fall outside [0, total_tokens] is treated as empty and the next carve_check returns
 * CARVE_ERR_INVALID_ARG (results are undefined, but nothing outside the buffers is touched).
 * Every packed call looks at its offsets, one without rows too.
 * With cu_seqlens NULL, tensors are [B, T, heads, channels] and total_tokens is ignored.
 *
 * Outputs overlap no input, except where a call says so.
 *
 * Inputs are expected to be finite.  A non-finite value reaches, beside the tokens that see it,
 * at most the other tokens of its own sequence that share a compute tile with them; it never
 * reaches another sequence.
 */
#ifndef CARVE_MIXERS_H
#define CARVE_MIXERS_H

#include "carve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the scalar-gated delta rule ----------------------------------------------------------
 * Per batch element (or sequence) and value head, a state S in R^{dv x dk}:
 *   a_t = exp(-e^{A_dec} softplus(g_logit_t + tau)),  w_t = sigmoid(w_logit_t)   (scalars)
 *   S_t = a_t S_{t-1} + w_t (v_t - a_t S_{t-1} k_t) k_t^T
 *   o_t = S_t q_t
 * the scalar-gated member of the delta-rule family that the CARVE recurrence generalises
 * (gist.science summary, Theorem 1).  Value heads share key heads in groups: value head h uses
 * key head h / (Hv / Hk).
 *
 *   q, k              [B, T, Hk, dk]  io       v, o              [B, T, Hv, dv]  io
 *   g_logit, w_logit  [B, T, Hv]      io       A_dec, tau        [Hv] float, nullable (0)
 *   S0, S_final       [B, Hv, dv, dk] float, nullable
 * Gradients have the layout and dtype of their tensor.  dk, dv in {64, 128}; Hv a multiple of
 * Hk; any T >= 0 (token pointers may be NULL when there are no rows).  Keys are meant to be
 * L2-normalised (the recurrence is contractive then); q is used as given (no scale).  A logit of any
 * finite size may reset the state: log decays below -1e4 count as -1e4, zero either way. */
typedef struct {
    int B, T, Hk, Hv, dk, dv;
    int io;                 /* carve_io */
    int64_t total_tokens;   /* rows of packed tensors (with cu_seqlens) */
} carve_gdr_dims;

/* Bytes of the forward's scratch, of the buffer it saves for carve_gdr_bwd, and of the
 * backward's scratch; `packed` tells whether the call passes cu_seqlens.  0 if the dims are
 * invalid. */
size_t carve_gdr_fwd_workspace_bytes(const carve_gdr_dims *d, int packed);
size_t carve_gdr_saved_bytes(const carve_gdr_dims *d, int packed);
size_t carve_gdr_bwd_workspace_bytes(const carve_gdr_dims *d, int packed);

/* Forward.  saved: NULL, or carve_gdr_saved_bytes for carve_gdr_bwd; workspace:
 * carve_gdr_fwd_workspace_bytes, NULL allowed when `saved` is given (its head serves).  S_final
 * may be S0 itself (the state updated in place). */
carve_status carve_gdr_fwd(const carve_gdr_dims *d, const int32_t *cu_seqlens, const void *q,
                           const void *k, const void *v, const void *g_logit, const void *w_logit,
                           const float *A_dec, const float *tau, const float *S0, void *o,
                           float *S_final, void *saved, void *workspace, void *stream);

/* Gradients of sum(dO * o) + sum(dS_final * S_final) with respect to every input.  The forward's
 * inputs and its `saved` buffer are passed unchanged.  dS_final (0 when NULL) and dS0 nullable;
 * A_dec with dA_dec and tau with dtau both NULL or both given ([Hv], summed over every token in
 * a fixed order).  Deterministic. */
carve_status carve_gdr_bwd(const carve_gdr_dims *d, const int32_t *cu_seqlens, const void *q,
                           const void *k, const void *v, const void *g_logit, const void *w_logit,
                           const float *A_dec, const float *tau, const void *saved, const void *dO,
                           const float *dS_final, void *dq, void *dk, void *dv, void *dg_logit,
                           void *dw_logit, float *dA_dec, float *dtau, float *dS0, void *workspace,
                           void *stream);

/* One token of every batch element (T and total_tokens are ignored): q, k [B, Hk, dk], v, o
 * [B, Hv, dv], g_logit, w_logit [B, Hv]; S [B, Hv, dv, dk] float read and written in place. */
carve_status carve_gdr_step(const carve_gdr_dims *d, const void *q, const void *k, const void *v,
                            const void *g_logit, const void *w_logit, const float *A_dec,
                            const float *tau, float *S, void *o, void *stream);

/* ---- sliding-window attention with sink tokens ----------------------------------------------
 * Query i of a sequence sees key j <= i where i - j < window or j < sinks:
 *   o_i = sum_j p_ij v_j,  p_i = softmax over the visible j of scale q_i . k_j
 * Query heads share key heads in groups: query head h uses key head h / (Hq / Hkv).
 *
 *   q, o   [B, T, Hq, d]  io      k, v  [B, T, Hkv, d]  io      lse  [rows, Hq] float
 * (lse: the natural logarithm of each row's softmax sum, with the scale).  d in {64, 128}; Hq a
 * multiple of Hkv; window >= 1; sinks >= 0; scale finite; any T >= 0. */
typedef struct {
    int B, T, Hq, Hkv, d;
    int window, sinks;
    int io;                 /* carve_io */
    float scale;
    int64_t total_tokens;   /* rows of packed tensors (with cu_seqlens) */
} carve_swa_dims;

/* Forward.  lse: nullable, needed by carve_swa_bwd. */
carve_status carve_swa_fwd(const carve_swa_dims *d, const int32_t *cu_seqlens, const void *q,
                           const void *k, const void *v, void *o, float *lse, void *stream);

/* Bytes of the backward's scratch (0 if the dims are invalid). */
size_t carve_swa_bwd_workspace_bytes(const carve_swa_dims *d, int packed);

/* Gradients of sum(dO * o) with respect to q, k and v, from the forward's inputs, o and lse.
 * Deterministic. */
carve_status carve_swa_bwd(const carve_swa_dims *d, const int32_t *cu_seqlens, const void *q,
                           const void *k, const void *v, const void *o, const float *lse,
                           const void *dO, void *dq, void *dk, void *dv, void *workspace,
                           void *stream);

/* The cache of the window, per batch element sinks + window slots: token t of a sequence lives
 * in slot t when t < sinks, else in slot sinks + (t - sinks) mod window, so that the slots hold
 * exactly the tokens that the next query sees.  k_cache, v_cache [B, sinks + window, Hkv, d] io.
 *
 * carve_swa_fill writes the tokens that stay visible after a prompt (the first `sinks` and the
 * last `window` ones of each sequence) into their slots; other slots are left as they were. */
carve_status carve_swa_fill(const carve_swa_dims *d, const int32_t *cu_seqlens, const void *k,
                            const void *v, void *k_cache, void *v_cache, void *stream);

/* One token of every batch element: q, o [B, Hq, d], k, v [B, Hkv, d]; pos [B] int64 DEVICE, the
 * tokens that each sequence already has (not changed; a negative one writes nothing to the
 * caches and yields zeros).  Writes k and v into the token's slot and attends to every visible
 * token, this one included.  T and total_tokens are ignored. */
carve_status carve_swa_step(const carve_swa_dims *d, const void *q, const void *k, const void *v,
                            void *k_cache, void *v_cache, const int64_t *pos, void *o, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CARVE_MIXERS_H */
