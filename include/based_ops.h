/*
 * based_ops.h: C ABI of the language-model operators around the Based forward pass (based.h):
 * the gated linear recurrence, the per-token group norm with an activation, the scaled
 * embedding with its gradient, the gated delta rule, the root-mean-square norm of a residual
 * stream and the choice of a next token.
 *
 * Conventions shared by every entry point (return codes, streams and error strings are those of
 * based.h):
 *   - Element types are given by a BASED_F32 / BASED_BF16 / BASED_F16 code. States, saved states
 *     and accumulations are float32 whatever the element type (based_delta_fwd says what it
 *     saves); each output element is rounded once, to nearest even.
 *   - The channel axis has stride 1. Other strides of inputs are arguments, in elements (a stride
 *     of 0 broadcasts, negative ones are refused); outputs are contiguous. Offsets are computed
 *     in 64 bits.
 *   - Pointers must be aligned to their element size. 16-byte aligned pointers with strides and
 *     sizes that keep rows 16-byte aligned take wider loads. In both norms and in based_delta_step
 *     the order in which sums are taken follows the loads, so that the same values at other strides
 *     or alignments can give other bits; elsewhere nothing but time depends on alignment.
 *   - Inputs are read-only. Outputs must not overlap inputs, except where stated.
 *   - Calls are asynchronous on `stream`, never synchronise and never allocate. Scratch, where an
 *     operator needs some, is a caller's workspace (16-byte aligned; contents ignored on entry,
 *     unspecified on return; calls that share one must not overlap on the GPU). Calls can be
 *     captured into CUDA graphs.
 *   - Results do not depend on timing: the same call on the same inputs gives the same bits.
 *   - Errors of arguments are detected on the host before anything is launched.
 */
#ifndef BASED_GB300_OPS_H
#define BASED_GB300_OPS_H

#include "based.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { BASED_F32 = 0, BASED_BF16 = 1, BASED_F16 = 2 };

/* How the recurrence turns its gate g and input x into a decay a and an increment u. */
enum {
    BASED_GATE_LOG = 0,    /* a = exp(g), u = x: g is the log decay (g = -inf clears the state; g > 0 makes it grow) */
    BASED_GATE_SIGMOID = 1 /* a = 1 / (1 + exp(-g)), u = (1 - a) x: g is the forget-gate logit */
};

/* Activations. */
enum { BASED_ACT_NONE = 0, BASED_ACT_SILU = 1, BASED_ACT_SIGMOID = 2 };

/* Rows between the states that based_scan_fwd saves for based_scan_bwd. */
#define BASED_SCAN_SAVE_ROWS 64

/*
 * based_scan_fwd: the gated linear recurrence
 *     h_t = a_t h_{t-1} + u_t,   t = 0 .. T-1, independently for each batch entry and channel,
 * with a and u from the gate and input by `mode`, computed and carried in float32.
 * States may be anything that float32 holds, row by row, with two exceptions. Where log gates add up
 * to more than 88 within sixteen rows (0-15, 16-31, ...), a state of 0 in front of them stays 0,
 * and one that is not 0 becomes infinite, however small it is. And what a tile of 64 rows or sixteen
 * of its rows would make of a state of 0 has to fit float32 too. A state that is infinite stays so,
 * or is NaN.
 *   gate, x      (B,T,D) of `dtype`, strides (gate_sb, gate_st, 1) and (x_sb, x_st, 1)
 *   state        (B,D) float32: h_{-1}; NULL is zero
 *   lengths      (B) int32 or NULL: rows t >= lengths[b] are padding: they leave the state as it
 *                is, their inputs are not read and their outputs are zero. Values are clamped to
 *                [0, T].
 *   y            (B,T,D) of `dtype`, contiguous: h_t
 *   final_state  (B,D) float32 or NULL: h after the last row; may be `state` itself
 *   saved        (B, ceil(T / BASED_SCAN_SAVE_ROWS), D) float32 or NULL: the states before rows
 *                0, 64, 128, ..., which based_scan_bwd reads
 * Errors: BASED_ERR_NULL_POINTER, BASED_ERR_UNSUPPORTED_TYPE, BASED_ERR_BAD_ARGUMENT (mode),
 * BASED_ERR_BAD_SIZE (B, T or D < 1, T > 2^30, D > 2^20 or B D >= 2^30), BASED_ERR_BAD_STRIDE, BASED_ERR_MISALIGNED,
 * BASED_ERR_ALIASING, BASED_ERR_CUDA, BASED_ERR_NO_DEVICE.
 */
BASED_API int based_scan_fwd(const void *gate, int64_t gate_sb, int64_t gate_st, const void *x, int64_t x_sb,
                             int64_t x_st, int B, int T, int D, int dtype, int mode, const float *state,
                             const int32_t *lengths, void *y, float *final_state, float *saved,
                             based_stream_t stream);

/*
 * based_scan_bwd: gradients of based_scan_fwd. With lam_t = dy_t + a_{t+1} lam_{t+1}, where the
 * row after the last contributes dfinal,
 *     BASED_GATE_LOG:      dgate = a_t h_{t-1} lam_t,                   dx = lam_t
 *     BASED_GATE_SIGMOID:  dgate = a_t (1 - a_t) (h_{t-1} - x_t) lam_t, dx = (1 - a_t) lam_t
 *     dstate = a_0 lam_0.
 * h is recomputed in float32 from the saved states, so that it is not a rounded one.
 *   gate, x, lengths, mode  as given to based_scan_fwd
 *   dy           (B,T,D) of `dtype`, strides (dy_sb, dy_st, 1); not read in padding rows
 *   saved        what based_scan_fwd wrote
 *   dfinal       (B,D) float32 or NULL (zero): gradient of final_state
 *   dgate, dx    (B,T,D) of `dtype`, contiguous; zero in padding rows
 *   dstate       (B,D) float32 or NULL
 * Errors: as based_scan_fwd.
 */
BASED_API int based_scan_bwd(const void *gate, int64_t gate_sb, int64_t gate_st, const void *x, int64_t x_sb,
                             int64_t x_st, const void *dy, int64_t dy_sb, int64_t dy_st, const float *saved, int B,
                             int T, int D, int dtype, int mode, const float *dfinal, const int32_t *lengths,
                             void *dgate, void *dx, float *dstate, based_stream_t stream);

/*
 * based_scan_step: one row of the recurrence for N sequences whose states lie in a pool:
 *     pool[s] = a pool[s] + u,  y_i = pool[s],   s = slots[i] (or i where slots is NULL).
 *   gate, x  (N,D) of `dtype`, row strides gate_sn and x_sn
 *   pool     (S,D) float32, contiguous, updated in place
 *   slots    (N) int32 or NULL (then S >= N). A slot outside [0, S) marks an idle row: no state
 *            changes and y_i is zero. No two rows may name the same slot (the result of that
 *            slot is then unspecified).
 *   y        (N,D) of `dtype`, contiguous
 * Errors: as based_scan_fwd.
 */
BASED_API int based_scan_step(const void *gate, int64_t gate_sn, const void *x, int64_t x_sn, int N, int D, int S,
                              int dtype, int mode, float *pool, const int32_t *slots, void *y,
                              based_stream_t stream);

/*
 * based_norm_fwd: group norm over the channels of each row, with an activation:
 *     v = (x - mean) / sqrt(var + eps) * weight + bias,   mean and var (biased) over the C / G
 *     consecutive channels of the element's group in its row;
 *     y = v act(gate)  where there is a gate,   y = act(v)  otherwise.
 * The statistics never mix rows, so a causal model stays causal. They are taken in two passes
 * over registers (the mean first, then the squared deviations), in float32.
 *   x       (R,C) of x_dtype, row stride x_sr
 *   gate    (R,C) of dtype, row stride gate_sr, or NULL
 *   weight, bias  (C) of p_dtype, each may be NULL (1 and 0)
 *   y       (R,C) of dtype, contiguous; may be `gate` or `x` itself where that is contiguous and
 *           of the same type
 *   dtype   is x_dtype, or any type where x_dtype is BASED_F32
 * C must be a multiple of G and at most 2^20, and C / G at most 4096.
 * Errors: as based_scan_fwd.
 */
BASED_API int based_norm_fwd(const void *x, int64_t x_sr, int x_dtype, const void *gate, int64_t gate_sr,
                             const void *weight, const void *bias, int p_dtype, int64_t R, int C, int G, float eps,
                             int act, void *y, int dtype, based_stream_t stream);

/*
 * based_norm_bwd: gradients of based_norm_fwd.
 *   dy       (R,C) of dtype, row stride dy_sr
 *   dx       (R,C) of x_dtype, contiguous
 *   dgate    (R,C) of dtype, contiguous; needed if and only if there is a gate
 *   dweight, dbias  (C) of p_dtype; each may be NULL. Sums over rows are taken in float32, in an
 *            order that depends on the sizes, types, strides, alignment and the GPU's number of SMs alone.
 *   workspace  based_norm_bwd_workspace_size() bytes (0 where dweight and dbias are NULL)
 * The statistics are recomputed from x. The rest as for based_norm_fwd.
 */
BASED_API int based_norm_bwd(const void *dy, int64_t dy_sr, const void *x, int64_t x_sr, int x_dtype,
                             const void *gate, int64_t gate_sr, const void *weight, const void *bias, int p_dtype,
                             int64_t R, int C, int G, float eps, int act, void *dx, void *dgate, void *dweight,
                             void *dbias, int dtype, void *workspace, size_t ws_bytes, based_stream_t stream);

/* Bytes of workspace based_norm_bwd() needs for these sizes, with dweight or dbias, on the
 * current device (0 for sizes it refuses). */
BASED_API size_t based_norm_bwd_workspace_size(int64_t R, int C, int G);

/*
 * based_embed_fwd: y_i = scale * table[ids[i]].
 *   ids     (N), int32, or int64 where ids64 is not 0. An id outside [0, V) is padding: its row
 *           of y is zero.
 *   table   (V,D) of dtype, row stride table_sr
 *   y       (N,D) of dtype, contiguous
 * Errors: as based_scan_fwd.
 */
BASED_API int based_embed_fwd(const void *ids, int ids64, const void *table, int64_t table_sr, int64_t N, int V,
                              int D, int dtype, float scale, void *y, based_stream_t stream);

/*
 * based_embed_bwd: dtable_v = scale * sum of dy_i over the i with ids[i] = v, in float32, in an
 * order that depends on the ids alone: the tokens are sorted by id (stably) and each id's rows
 * are summed in tiles of the sorted order. Rows of ids that do not occur are set to zero.
 *   dy      (N,D) of dtype, row stride dy_sr
 *   dtable  (V,D) of g_dtype (dtype or BASED_F32), contiguous
 *   workspace  based_embed_bwd_workspace_size() bytes
 * N must be below 2^30 and D at most 2^20.
 */
BASED_API int based_embed_bwd(const void *ids, int ids64, const void *dy, int64_t dy_sr, int64_t N, int V, int D,
                              int dtype, float scale, void *dtable, int g_dtype, void *workspace, size_t ws_bytes,
                              based_stream_t stream);

/* Bytes of workspace based_embed_bwd() needs for these sizes (0 for sizes it refuses). */
BASED_API size_t based_embed_bwd_workspace_size(int64_t N, int V, int D);

/*
 * based_delta_fwd: the gated delta rule, a linear attention whose state (K,V) decays and corrects what it
 * has stored: per batch entry and head, for t = 0 .. T-1,
 *     u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   S_t = a_t S_{t-1} + k_t u_t^T,   o_t = scale S_t^T q_t,
 * with a = exp(gate), or 1 without gates. Head h of the values uses head h / (H / HK) of queries and keys.
 * Products go through pairs of float16 terms, scaled by the largest magnitude of 16 value channels of the state, of 64 rows of keys, of queries
 * or of their products, and of 16 rows by 16 channels of values (a row counts times |beta|, or 2^-12 where that is less) and of their gradients: off
 * by 2^-22 of a number down to 2^-17 of the largest that it shares its scale with, and by 2^-39 of that below. Sums are float32's.
 * Where `dtype` is BASED_BF16, what is in outputs and gradients alone is one term, off by 2^-11 of a number where the result's rounding is off by
 * 2^-8: the state as q reads it, scores and corrections, and backward also what `saved` holds. What goes into a state is a pair.
 * Magnitudes below 2^-84 count as 0, and from 2^115 on as infinite.
 * Gates are meant to be <= 0 (-inf clears the state, gates below -1e5 count as -inf). Positive ones let the state grow and
 * work as long as no 64 of them add up to more than 88. Rows go by chunks of 64, from row 0: from the chunk on that has an
 * infinity or NaN in an input or the state, a head's results are NaN where the formulas have them, and undefined elsewhere.
 * Keys are taken as they are; the rule is stable where beta |k|^2 is at most 2.
 *   q, k         (B,T,HK,K) of `dtype`, strides (sb, st, sh, 1)
 *   v            (B,T,H,V) of `dtype`, strides (sb, st, sh, 1)
 *   beta, gate   (B,T,H) of `dtype`, strides (sb, st, 1); gate may be NULL
 *   scale        <= 0 selects K^-0.5
 *   state        (B,H,K,V) float32: S_{-1}; NULL is zero
 *   lengths      (B) int32 or NULL: rows t >= lengths[b] are padding: they leave the state as it is, their
 *                inputs are not read and their outputs are zero. Values are clamped to [0, T].
 *   o            (B,T,H,V) of `dtype`, contiguous
 *   final_state  (B,H,K,V) float32 or NULL: S_{T-1}; may be `state` itself
 *   saved        based_delta_saved_size() bytes, 16-byte aligned, or NULL: what based_delta_bwd reads (the states in front of rows 0, 64, ...
 *                and the rows' v_t - a_t S_{t-1}^T k_t, as float16 terms in the kernels' own order: two a number, one in bfloat16)
 *   workspace    based_delta_workspace_size(..., 0) bytes
 * H must be a multiple of HK, K at most 128, V at most 65536.
 * Errors: as based_scan_fwd, BASED_ERR_WORKSPACE, BASED_ERR_BAD_ARGUMENT (a scale that is NaN).
 */
BASED_API int based_delta_fwd(const void *q, int64_t q_sb, int64_t q_st, int64_t q_sh, const void *k, int64_t k_sb,
                              int64_t k_st, int64_t k_sh, const void *v, int64_t v_sb, int64_t v_st, int64_t v_sh,
                              const void *beta, int64_t beta_sb, int64_t beta_st, const void *gate, int64_t gate_sb,
                              int64_t gate_st, int B, int T, int H, int HK, int K, int V, int dtype, float scale,
                              const float *state, const int32_t *lengths, void *o, float *final_state, void *saved,
                              void *workspace, size_t ws_bytes, based_stream_t stream);

/*
 * based_delta_bwd: gradients of based_delta_fwd for the gradients dout (B,T,H,V) of o and dfinal of final_state.
 * Queries' and keys' gradients are summed over the heads that share them, in a fixed order.
 *   q .. gate, scale, lengths  as given to based_delta_fwd
 *   dout         (B,T,H,V) of `dtype`, strides (do_sb, do_st, do_sh, 1); not read in padding rows
 *   saved        what based_delta_fwd wrote
 *   dfinal       (B,H,K,V) float32 or NULL (zero)
 *   dq, dk       (B,T,HK,K), dv (B,T,H,V), dbeta, dgate (B,T,H) of `dtype`, contiguous, zero in padding rows;
 *                dgate if and only if there are gates; dq and dk aligned to two elements
 *   dstate       (B,H,K,V) float32 or NULL
 *   workspace    based_delta_workspace_size(..., 1) bytes
 * Errors: as based_delta_fwd.
 */
BASED_API int based_delta_bwd(const void *q, int64_t q_sb, int64_t q_st, int64_t q_sh, const void *k, int64_t k_sb,
                              int64_t k_st, int64_t k_sh, const void *v, int64_t v_sb, int64_t v_st, int64_t v_sh,
                              const void *beta, int64_t beta_sb, int64_t beta_st, const void *gate, int64_t gate_sb,
                              int64_t gate_st, const void *dout, int64_t do_sb, int64_t do_st, int64_t do_sh,
                              const void *saved, int B, int T, int H, int HK, int K, int V, int dtype,
                              float scale, const float *dfinal, const int32_t *lengths, void *dq, void *dk,
                              void *dv, void *dbeta, void *dgate, float *dstate, void *workspace, size_t ws_bytes,
                              based_stream_t stream);

/* Bytes of workspace based_delta_fwd() (backward 0) or based_delta_bwd() needs for these sizes (0 for sizes they refuse). */
BASED_API size_t based_delta_workspace_size(int B, int T, int H, int HK, int K, int V, int dtype, int backward);

/* Bytes that based_delta_fwd() saves for based_delta_bwd() (0 for sizes they refuse). */
BASED_API size_t based_delta_saved_size(int B, int T, int H, int K, int V, int dtype);

/*
 * based_delta_step: one row of the delta rule for N sequences whose states lie in a pool:
 *     S = a pool[s],  u = beta (v - S^T k),  pool[s] = S + k u^T,  o_i = scale pool[s]^T q,   s = slots[i] (or i).
 *   q, k (N,HK,K) and v (N,H,V) of `dtype`, strides (sn, sh, 1); beta, gate (N,H), strides (sn, 1); gate may be NULL
 *   pool     (S,H,K,V) float32, contiguous, updated in place
 *   slots    as for based_scan_step
 *   o        (N,H,V) of `dtype`, contiguous
 * Errors: as based_delta_fwd.
 */
BASED_API int based_delta_step(const void *q, int64_t q_sn, int64_t q_sh, const void *k, int64_t k_sn, int64_t k_sh,
                               const void *v, int64_t v_sn, int64_t v_sh, const void *beta, int64_t beta_sn,
                               const void *gate, int64_t gate_sn, int N, int H, int HK, int K, int V, int S, int dtype,
                               float scale, float *pool, const int32_t *slots, void *o, based_stream_t stream);

/*
 * based_rms_fwd: root-mean-square norm of a residual stream, with the addition in front of it:
 *     s = x + residual, rounded to s_dtype (or s = x),   y = s / sqrt(mean(s^2) + eps) * weight,
 * the mean over the C channels of a row. The norm is that of the s that is written. Squares are summed in float32: a row whose sum passes it
 * (magnitudes of some 2^60) has an infinite size.
 *   x         (R,C) of dtype, row stride x_sr
 *   residual  (R,C) of s_dtype (dtype or BASED_F32), row stride res_sr, or NULL
 *   weight    (C) of p_dtype (dtype or BASED_F32), or NULL (1)
 *   sum       (R,C) of s_dtype, contiguous: s; NULL if and only if there is no residual; may be `residual` where that is contiguous
 *   y         (R,C) contiguous, of dtype; or, where scales are given, e4m3 bytes (one an element):
 *             y = y8 * scales[row] with scales[row] = max|y| / 448 (1 for a row of zeros), rounded to nearest even
 *   scales    (R) float32 or NULL
 * C is at most 16384. Errors: as based_scan_fwd.
 */
BASED_API int based_rms_fwd(const void *x, int64_t x_sr, const void *residual, int64_t res_sr, int s_dtype,
                            const void *weight, int p_dtype, int64_t R, int C, float eps, void *sum, void *y, int dtype,
                            float *scales, based_stream_t stream);

/*
 * based_rms_bwd: gradients of based_rms_fwd (its output of dtype).
 *   dy       (R,C) of dtype, row stride dy_sr
 *   s        the sum that based_rms_fwd wrote (without a residual its x), (R,C) of s_dtype, row stride s_sr
 *   dsum     (R,C) of s_dtype, row stride dsum_sr: what comes back along the stream, added to ds; or NULL
 *   ds       (R,C) of s_dtype, contiguous: the gradient of the residual (and of x); may be `dsum` where that is contiguous
 *   dx       (R,C) of dtype, contiguous: ds in the type of x; NULL if and only if s_dtype is dtype
 *   dweight  (C) of p_dtype or NULL; summed in float32 in an order that sizes and alignment fix
 *   workspace  based_rms_bwd_workspace_size() bytes (none where dweight is NULL)
 * Errors: as based_rms_fwd, BASED_ERR_WORKSPACE.
 */
BASED_API int based_rms_bwd(const void *dy, int64_t dy_sr, const void *s, int64_t s_sr, int s_dtype, const void *weight,
                            int p_dtype, const void *dsum, int64_t dsum_sr, int64_t R, int C, float eps, void *ds,
                            void *dx, void *dweight, int dtype, void *workspace, size_t ws_bytes,
                            based_stream_t stream);

/* Bytes of workspace based_rms_bwd() needs for these sizes, with dweight (0 for sizes it refuses). */
BASED_API size_t based_rms_bwd_workspace_size(int64_t R, int C);

/*
 * based_sample: the next token of each row of logits, from given random numbers. Tokens are ordered by falling logits, equal ones
 * by rising index; with p_i the softmax of logits / temperature, a row keeps
 *     the first top_k of the order; of these the fewest of the first whose p reach the share top_p of theirs;
 *     and of these the ones with p_i >= min_p max(p),
 * and takes, in the order of indices, the first whose kept p sum up to more than u times the sum of all kept ones.
 *   logits       (N,V) of dtype, row stride `stride`. -inf is never taken, NaN counts as -inf. A row of -inf gives token -1 and
 *                probability 0; a row with +inf its first +inf.
 *   u            (N) float32 in [0, 1)
 *   temperature, top_k, top_p, min_p  (N) float32 (top_k int32), one for each row, or NULL: then the value behind it holds for all rows.
 *                temperature <= 0 takes the first of the order; top_k <= 0, top_p >= 1 and min_p <= 0 keep all; top_p <= 0 keeps the first; NaN keeps all
 *                (as a temperature: the first).
 *   tokens       (N) int32
 *   probs        (N) float32 or NULL: the token's share of what its row keeps
 * Probabilities are computed in float32 (to 2^-21) and summed as whole multiples of 2^-40 of the largest, eight neighbours at a time: tokens below that
 * have none. A row's token and probability depend on the row alone, not on the others of the call nor on alignment.
 * V is at most 2^22, N at most 2^26. Errors: as based_scan_fwd.
 */
BASED_API int based_sample(const void *logits, int64_t stride, int dtype, int N, int V, const float *u,
                           const float *temperature, float temperature_all, const int32_t *top_k, int top_k_all,
                           const float *top_p, float top_p_all, const float *min_p, float min_p_all, int32_t *tokens,
                           float *probs, based_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BASED_GB300_OPS_H */
