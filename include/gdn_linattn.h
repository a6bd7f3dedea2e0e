/*
 * gdn_linattn.h -- C ABI of the operators beside the gated delta rule (gdn.h):
 * linear attention with a decay for each head, the norm and rotation of queries
 * and keys, and beam search over recurrent states, on NVIDIA B200 (sm_100a).
 *
 * Conventions are those of gdn.h: device pointers owned by the caller, no device
 * memory allocated by the library, calls asynchronous on `stream`, argument errors
 * found on the host before anything is launched (all outputs untouched), the reason
 * of a failure in gdn_last_error().  Every call may be captured into a CUDA graph.
 */
#ifndef GDN_LINATTN_H_
#define GDN_LINATTN_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A third gate kind, for gdn_desc.gate of the gdn_linattn_* calls only: one fixed
 * decay per head, log_gate (H) fp32, the same for every token and sequence. */
enum { GDN_GATE_CONST = 2 };

/* ---------------------------------------------------------------------------
 * Linear attention with a decay for each head: the recurrence of gdn.h without the
 * delta correction,
 *
 *     S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = S_t (scale q_t),   alpha = exp(log_gate)
 *
 * with S a d_v x d_k fp32 state per sequence and value head, in the state layout of
 * gdn.h.  d->gate is GDN_GATE_HEAD (log_gate (B, T, H): a decay per head and token)
 * or GDN_GATE_CONST (log_gate (H)); GDN_GATE_CHANNEL is GDN_ERR_UNSUPPORTED.
 * log_gate holds values <= 0 (0: no decay; -105 or less, -infinity too: the state is
 * erased); sizes, dtypes, shared query/key heads and alignment as in gdn.h.  q, k and v
 * hold finite values: a value that is
 * not finite makes the outputs of its 64-token chunk and of everything after it in
 * its sequence and head unspecified (other sequences and heads are not affected), and so
 * do sums of |q . k| |v| over a chunk of 2^67 or more (bf16, 128-wide heads).
 *
 * Precision.  States are fp32 sums of unrounded products: within 1e-5 (relative) over hundreds
 * of thousands of tokens that do not fade, below 1e-6 as a rule.  Outputs are rounded once from
 * fp32 sums, but for bf16 prompts with 128-wide heads (gdn_linattn_chunk_fwd, on the tensor
 * cores): there the scores q . k, with their decays, and the state that meets q are rounded to
 * bf16 first, once each, and where a chunk's decay is below 2^-120 the q that meets the state
 * once more; outputs are then within 3 * 2^-8 (relative to their head's length; 2.3e-3 is
 * usual, against 1.7e-3 for the last rounding alone), and contributions |q . k| |v| of less
 * than 2^-64 may be lost.
 * ------------------------------------------------------------------------- */

/* Bytes of device workspace gdn_linattn_chunk_fwd needs for d->T tokens in num_seqs
 * sequences (B when cu_seqlens is NULL); covers any packing and both gate kinds. */
gdn_status gdn_linattn_workspace_size(const gdn_desc *d, int32_t num_seqs, size_t *bytes);

/* ---------------------------------------------------------------------------
 * gdn_linattn_chunk_fwd -- prompts, by the chunkwise form.
 *
 * Arguments as gdn_chunk_fwd (gdn.h) without beta: fixed-length sequences or packed
 * ones (cu_seqlens, B == 1), initial and final states, snapshots every
 * snapshot_stride tokens (a multiple of 64; not with cu_seqlens).  final_state may be
 * initial_state.  Offsets in cu_seqlens are read on the device and not validated there:
 * wrong offsets give wrong results, but every access stays inside the B*T rows.  Rows
 * of `out` outside every sequence are not written.  Every sequence's result depends on
 * its own tokens only.  Long sequences are split into segments that run side by side;
 * a token whose decay to a segment's end is below 2^-149 does not reach it.
 *
 * The first 4 bytes of the workspace hold the call's device status, read with
 * gdn_chunk_status (GDN_DEV_TIMEOUT_PREP: the kernel of the segments' states,
 * GDN_DEV_TIMEOUT_SCAN: the kernel of the outputs).  Two calls in flight at once need
 * two workspaces; calls (or replays of captured ones) that share one run one after
 * the other on one stream.
 * ------------------------------------------------------------------------- */
gdn_status gdn_linattn_chunk_fwd(const gdn_desc *d,
                                 const void *q, const void *k, const void *v, const float *log_gate,
                                 const float *initial_state,
                                 const int32_t *cu_seqlens, int32_t num_seqs, int64_t snapshot_stride,
                                 void *out, float *final_state, float *snapshots,
                                 void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* ---------------------------------------------------------------------------
 * gdn_linattn_decode_step -- one token of every live sequence (d->T == 1), the state
 * updated in place: S' = alpha S + v k^T, o = S' (scale q) = alpha S (scale q) + v (k . scale q).
 *   q, k (B, 1, hk, d_k); v, out (B, 1, H, d_v); log_gate (B, 1, H), or (H) for
 *   GDN_GATE_CONST; state (B, H, d_v, d_k), read and overwritten.  Errors as
 *   gdn_decode_step.
 * ------------------------------------------------------------------------- */
gdn_status gdn_linattn_decode_step(const gdn_desc *d, const void *q, const void *k, const void *v,
                                   const float *log_gate, float *state, void *out, gdn_stream_t stream);

/* ---------------------------------------------------------------------------
 * gdn_qk_norm_rope -- the norm of every query and key head and the position rotation,
 * in one pass over them: for every token and head x (head_dim values),
 *
 *     y = x / sqrt(mean(x^2) + eps) * (weight_offset + weight)
 *     (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position inv_freq[i]
 *
 * for i < rot / 2, where (a, b) = (i, i + rot / 2), or (2 i, 2 i + 1) when
 * `interleaved`; channels from rot on are not rotated.  The norm and the rotation are in
 * fp32, the angle is formed and reduced in 64 bits (exact to fp32 up to a position times
 * inv_freq of 2^27, negative ones too; within 2^-20 up to 2^31), and the result is rounded once.
 * ------------------------------------------------------------------------- */
typedef struct gdn_qk_rope_desc {
    int64_t rows;       /* tokens (B * T)                                               */
    int32_t hq, hk;     /* query and key heads per token (hk may be 0: queries only)    */
    int32_t head_dim;   /* 64, 128 or 256                                               */
    int32_t rot;        /* rotated channels: 0, or a multiple of 16 up to head_dim      */
    int32_t interleaved;
    int32_t dtype;      /* gdn_dtype of q, k and the outputs                            */
    int64_t q_stride, k_stride; /* elements from a token's row of heads to the next one's
                                   (q and k may be slices of a wider projection); a
                                   multiple of 16 bytes                                 */
    float eps, weight_offset;
} gdn_qk_rope_desc;

/*   q, k          (rows) rows of (hq, head_dim) and (hk, head_dim), strides above, 16-byte aligned
 *   positions     (rows) int32 (may be NULL when rot == 0)
 *   inv_freq      (rot / 2) fp32 (may be NULL when rot == 0)
 *   q_weight, k_weight (head_dim) fp32, or NULL: all ones (weight_offset then unused)
 *   q_out, k_out  (rows, hq, head_dim), (rows, hk, head_dim) dense, 16-byte aligned; each
 *                 may be its input when that is dense, and overlaps nothing else         */
gdn_status gdn_qk_norm_rope(const gdn_qk_rope_desc *d, const void *q, const void *k, const int32_t *positions,
                            const float *inv_freq, const float *q_weight, const float *k_weight,
                            void *q_out, void *k_out, gdn_stream_t stream);

/* ---------------------------------------------------------------------------
 * gdn_beam_select -- one step of beam search: for each of B requests the K best of its
 * W * V continuations by
 *
 *     score[b, w, t] = scores[b, w] + logits[b, w, t] - log sum_u exp(logits[b, w, u]),
 *
 * best first; among equal scores the lowest w * V + t comes first (within a beam the
 * order is that of its logits).  A beam whose scores entry or whose sum is not finite (a
 * NaN or +infinite logit, no logit above -infinity, a finished beam marked with -infinity)
 * has all its scores at -infinity; continuations at -infinity come last, in index
 * order, and keep -infinity as their score.  Exponentials, and their sums over up to
 * 16,384 logits, are fp32; these sums are joined, and the scores formed and compared, in 64
 * bits and rounded once.  A beam's log-sum is within 2^-17 (2^-22 is usual), the same for
 * all its continuations: continuations of different beams whose scores are nearer than
 * that may come in either order (beams with the same logits at the same places have the same
 * log-sum).
 * ------------------------------------------------------------------------- */
typedef struct gdn_beam_desc {
    int64_t B;          /* requests                                                     */
    int32_t W;          /* beams per request, 1 .. 64                                   */
    int32_t V;          /* vocabulary, W * V < 2^31                                     */
    int32_t K;          /* continuations to keep per request, 1 .. min(64, W * V)       */
    int32_t dtype;      /* gdn_dtype of the logits                                      */
    int64_t row_stride; /* elements from a beam's logits to the next beam's, >= V       */
} gdn_beam_desc;

/* Bytes of device workspace gdn_beam_select needs. */
gdn_status gdn_beam_workspace_size(const gdn_beam_desc *d, size_t *bytes);

/*   logits      (B * W) rows of V values, row_stride apart (any element alignment)
 *   scores      (B, W) fp32, the beams' summed log-probabilities (NULL: zeros)
 *   out_scores  (B, K) fp32; out_parent, out_token (B, K) int32: the beam a continuation
 *               extends and its token
 *   workspace   gdn_beam_workspace_size bytes, 256-byte aligned, contents do not matter;
 *               two calls in flight at once need two                                     */
gdn_status gdn_beam_select(const gdn_beam_desc *d, const void *logits, const float *scores, float *out_scores,
                           int32_t *out_parent, int32_t *out_token, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream);

/* ---------------------------------------------------------------------------
 * gdn_state_reorder -- move per-beam rows to the beams that go on with them, in place:
 * row (b, w) <- row (b, parent[b, w]) for every request b and beam w, all rows read
 * as they were before the call.  A recurrent state has no pages that beams could
 * share, so after gdn_beam_select every beam takes its parent's state (and
 * convolution history): only rows that change are written, and only their parents
 * read.  A parent outside 0 .. W - 1 leaves its row as it is.
 *   state      (B, W) rows of row_bytes bytes, 16-byte aligned; row_bytes a multiple of 16
 *   parent     (B, W) int32, not inside the state;  W in 1 .. 64
 * ------------------------------------------------------------------------- */
gdn_status gdn_state_reorder(void *state, const int32_t *parent, int64_t B, int32_t W, size_t row_bytes,
                             gdn_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_LINATTN_H_ */
