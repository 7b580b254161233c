/*
 * based_ops.h: C ABI of the language-model operators around the Based forward pass (based.h):
 * the gated linear recurrence, the per-token group norm with an activation, and the scaled
 * embedding with its gradient.
 *
 * Conventions shared by every entry point (return codes, streams and error strings are those of
 * based.h):
 *   - Element types are given by a BASED_F32 / BASED_BF16 / BASED_F16 code. States, saved states
 *     and accumulations are float32 whatever the element type; each output element is rounded
 *     once, to nearest even.
 *   - The channel axis has stride 1. Other strides of inputs are arguments, in elements (a stride
 *     of 0 broadcasts, negative ones are refused); outputs are contiguous. Offsets are computed
 *     in 64 bits.
 *   - Pointers must be aligned to their element size. 16-byte aligned pointers with strides and
 *     sizes that keep rows 16-byte aligned take wider loads. In the norm the order in which sums are
 *     taken follows the loads, so that the same values at other strides or alignments can give
 *     other bits; in the other operators nothing but time depends on alignment.
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

#ifdef __cplusplus
}
#endif

#endif /* BASED_GB300_OPS_H */
