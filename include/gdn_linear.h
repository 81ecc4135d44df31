/*
 * gdn_linear.h -- C ABI of the gated linear recurrence on one GB300 GPU: the
 * diagonal-state sibling of the gated delta rule (gdn_prefill.h), on the same
 * packed variable-length batches and the same kind of state pool.
 *
 * The operation: for every sequence i of the packed batch and every channel c
 * (c = h * D + d, head h of H, D channels a head),
 *
 *     u_t = b_t x_t                       (without b: u_t = x_t)
 *     h_t = a_t h_{t-1} + u_t             h before the first token: the
 *     y_t = h_t                           initial state, or zero
 *
 * States and all arithmetic are fp32; y is rounded once, to x's type.
 *
 * Backward, from dy and (optionally) the gradient of the final state: with
 * the carry c_t = a_t g_t and g_t = dy_t + c_{t+1}, where c past the last
 * token of a sequence is d_final_state (or zero),
 *
 *     dx_t = b_t g_t    db_t = x_t g_t    da_t = h_{t-1} g_t
 *     d_initial_state = c at the sequence's first token
 *
 * with da and db summed over a head's channels when the gates are per head.
 * h_{t-1} is recomputed in fp32 from tile_states, which the forward run saves.
 *
 * Shapes (device memory):
 *   x, y, dy, dx      [T, H, D] in x_dtype: H * D contiguous elements a
 *                     token, *_stride elements from token to token (0: H * D)
 *   a, b, da, db      [T, H, D], or [T, H] with GDN_LINEAR_GATES_PER_HEAD, in
 *                     gate_dtype (x_dtype or F32), contiguous within a token,
 *                     strides as above (0: dense)
 *   cu_seqlens        [N+1] int32 or int64, cu_seqlens[0] = 0,
 *                     cu_seqlens[N] = T, equal neighbours are empty sequences;
 *                     NULL with num_seqs = 1: one sequence of T tokens
 *   initial_state,    [N, H, D], or a pool [n_pool, H, D] with state_indices,
 *   output_state      in state_dtype (F32, BF16, F16, F8E4M3 or F8E5M2; widened
 *                     on load, rounded to nearest on store), H * D contiguous
 *                     elements a row, state_stride elements from row to row
 *                     (0: dense); both may be one buffer
 *   tile_states       [ceil(T / 64), H, D] fp32, dense: row f is the state
 *                     after packed token min(64 f + 63, T - 1)
 *   d_final_state,    [N, H, D] fp32, dense
 *   d_initial_state
 * An empty sequence's final state is its initial state, and its
 * d_initial_state its d_final_state.
 *
 * Gates may have any value.  The scan forms products of the a of up to 64
 * successive tokens in fp32; these have to stay finite, which |a| < 4
 * guarantees, and bits of them that fall below 2^-149 are lost.  Products over
 * longer stretches have an exponent of their own.  The error of a result is
 * that of a sum of its terms' absolute values, which has to stay finite as
 * well.  A state that is not finite stays within its own sequence.
 * y may be x itself (same stride); other overlaps of outputs with inputs are
 * not allowed, except output_state with initial_state.
 *
 * Results do not depend on timing: the same inputs give the same bits.
 *
 * Ownership, streams and errors are those of gdn_prefill.h: the caller owns
 * every tensor and the workspace, runs only enqueue work on the caller's
 * stream, what the host can check is refused before anything is launched, and
 * device data is checked on the device (bits GDN_DEVICE_ERR_CU_SEQLENS,
 * GDN_DEVICE_ERR_STATE_INDEX_RANGE and GDN_DEVICE_ERR_TIMEOUT are OR-ed into
 * args.device_status, when it is given; the outputs are then unspecified).  A
 * state index outside [0, n_pool) is not followed.  Two sequences that name
 * one pool row race on it.  Waits of one block for another, or for its copies,
 * have a limit of one to four seconds.  After one that ran out
 * (GDN_DEVICE_ERR_TIMEOUT) the run ends, and outputs and states that depend
 * on what did not come are NaN, with device_status or without it.
 */
#ifndef GDN_LINEAR_H
#define GDN_LINEAR_H

#include "gdn_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_LINEAR_TILE 64 /* packed tokens a row of tile_states stands for */

/* gdn_linear_desc.flags */
enum {
    GDN_LINEAR_HAS_B = 1u << 0,
    GDN_LINEAR_GATES_PER_HEAD = 1u << 1,
    GDN_LINEAR_HAS_INITIAL_STATE = 1u << 2,
    GDN_LINEAR_OUTPUT_FINAL_STATE = 1u << 3,
    GDN_LINEAR_HAS_STATE_INDICES = 1u << 4,
    GDN_LINEAR_CU_SEQLENS_I64 = 1u << 5,
    GDN_LINEAR_STATE_INDICES_I64 = 1u << 6
};

typedef struct gdn_linear_desc {
    int32_t num_heads, head_dim; /* H, D >= 1; H * D <= 2^20 */
    gdn_dtype x_dtype;           /* BF16, F16 or F32 */
    gdn_dtype gate_dtype;        /* x_dtype or F32 */
    gdn_dtype state_dtype;       /* initial / output states */
    int64_t max_total_tokens;    /* upper bound of T over the plan's runs */
    int32_t max_num_seqs;        /* upper bound of N */
    uint32_t flags;              /* GDN_LINEAR_* */
} gdn_linear_desc;

typedef struct gdn_linear_plan_s *gdn_linear_plan_t;

typedef struct gdn_linear_args {
    const void *x, *a, *b;
    int64_t x_stride, a_stride, b_stride; /* elements from token to token; 0 = dense */
    const void *cu_seqlens;
    int32_t num_seqs;
    int64_t total_tokens;
    const void *initial_state;
    void *output_state;
    int64_t state_stride; /* elements from row to row; 0 = dense */
    const void *state_indices;
    int32_t n_pool;
    int32_t *device_status; /* optional */
    /* forward and decode */
    void *y;
    int64_t y_stride;
    float *tile_states; /* forward: optional output; backward: input, required when T > 64 */
    /* backward */
    const void *dy;
    int64_t dy_stride;
    const float *d_final_state; /* optional */
    float *d_initial_state;     /* optional */
    void *dx, *da, *db;         /* dx and da required; db with GDN_LINEAR_HAS_B */
    int64_t dx_stride, da_stride, db_stride;
} gdn_linear_args;

/* Validate `desc`, create a plan and say how large a workspace (16-byte
 * aligned device memory) its forward and backward runs need.  Needs no GPU.
 * A workspace serves one run at a time. */
gdn_status gdn_linear_plan(const gdn_linear_desc *desc, gdn_linear_plan_t *plan, size_t *workspace_bytes);
void gdn_linear_plan_destroy(gdn_linear_plan_t plan);

/* Bytes of workspace that the forward (backward != 0: the backward) run of
 * these arguments needs on the current device: at most the plan's, and 0 for
 * many (their workspace may be NULL).  0 for arguments that the run refuses. */
size_t gdn_linear_run_workspace(gdn_linear_plan_t plan, const gdn_linear_args *args, int32_t backward);

gdn_status gdn_linear_forward_run(gdn_linear_plan_t plan, const gdn_linear_args *args, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Gradients.  State pools are a matter of serving: the plan has no
 * state_indices (GDN_ERR_UNSUPPORTED). */
gdn_status gdn_linear_backward_run(gdn_linear_plan_t plan, const gdn_linear_args *args, void *workspace,
                                   size_t workspace_bytes, void *stream);

/* Decode: N sequences of exactly tokens_per_seq >= 1 tokens, token j of
 * sequence i at row i * tokens_per_seq + j; cu_seqlens, tile_states and the
 * workspace are not used.  T = N * tokens_per_seq. */
gdn_status gdn_linear_decode_run(gdn_linear_plan_t plan, const gdn_linear_args *args, int32_t tokens_per_seq,
                                 void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LINEAR_H */
