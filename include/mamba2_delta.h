/*
 * mamba2_delta.h -- C ABI of the gated delta rule and of the group norm beside
 * it, for AMD Instinct MI355X (gfx950).  Part of libmamba2scan.so, beside the
 * selective layer of mamba2_layer.h, whose types, conventions (memory, streams,
 * graphs, overlaps, refusals, reproducible results) and status codes it shares;
 * mamba2_layer_strerror names the codes.
 */
#ifndef MAMBA2_DELTA_H
#define MAMBA2_DELTA_H

#include "mamba2_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Gated delta rule.  Per sequence and head h, with the state S [states][width]
 * (fp32) and j = h / (heads / groups):
 *   S'     = e^(g_t[h]) S_{t-1}
 *   S_t    = S' + k_t[j] (beta_t[h] (v_t[h] - S'^T k_t[j]))^T
 *   y_t[h] = scale S_t^T q_t[j]
 *   q, k [groups][states], v, y [heads][width], g, beta [heads] per token;
 *   states' layout [batch][heads][states][width].
 * S_0 = initial_state (NULL: 0); final_state (NULL: skipped) gets the state
 * after the last token, and initial_state itself for an empty sequence.
 * A token whose g and beta are 0 leaves the state as it was; so a padded batch
 * marks its padding, q, k and v there being finite.  g = -inf forgets the state
 * before the token.
 *   g <= 0 is meant, and beta |k|^2 <= 2 (keys of length one, say: the group norm
 *   with a weight of width^-1/2), beyond which the recurrence itself grows; growing
 *   states are computed as long as e^(sum of g) over 64 tokens, and what the rule
 *   makes of the keys within them, stay finite.
 *   1 <= groups, heads a multiple of groups, at most 65535, as batch is;
 *   width and states multiples of 8, 8 .. 128.  q, k, v, y and the states are
 *   16-byte aligned, with row and batch strides that are multiples of 8
 *   elements; g and beta have any stride.  Row strides are at most 2^29 / 65
 *   elements.  A call has 512 threads for every step of 64 tokens and head, and
 *   for every sequence (a cut one: segment), head, 64 columns and 64 states.
 *   A value that is not finite may reach every token of its own sequence and
 * head (q, k: group) from the start of its step of 64 tokens on (gradients: up
 * to the end of it and before), but no other sequence; an infinity may come
 * out as a NaN.
 */
typedef struct {
  int type;       /* of q, k, v, y and their gradients                      */
  int gate_type;  /* of g and beta and their gradients                      */
  int heads;
  int width;      /* elements of a value (V)                                */
  int groups;     /* heads / groups neighbouring heads share one q and k    */
  int states;     /* elements of a query or key (K)                         */
  float scale;    /* of the results                                         */
} mamba2_delta_dims;

/* Bytes of the forward's workspace (each step's matrices); 0 for dimensions
 * that are refused. */
size_t mamba2_delta_fwd_workspace_bytes(mamba2_seqs seqs, mamba2_delta_dims dims);

int mamba2_delta_fwd(mamba2_seqs seqs, mamba2_delta_dims dims, mamba2_rows q,
                     mamba2_rows k, mamba2_rows v, mamba2_rows g,
                     mamba2_rows beta, const float* initial_state,
                     mamba2_rows y, float* final_state, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Bytes of the backward's workspace: each step's matrices, the states and
 * their gradients at the steps' borders; 0 for dimensions that are refused. */
size_t mamba2_delta_bwd_workspace_bytes(mamba2_seqs seqs, mamba2_delta_dims dims);

/*
 * Gradients for given dL/dy and, when not NULL, dL/dfinal_state.  The states
 * are recomputed from the inputs, which are given again.  d_q .. d_beta are
 * required; d_initial_state may be NULL.
 */
int mamba2_delta_bwd(mamba2_seqs seqs, mamba2_delta_dims dims, mamba2_rows q,
                     mamba2_rows k, mamba2_rows v, mamba2_rows g,
                     mamba2_rows beta, const float* initial_state,
                     mamba2_rows d_y, const float* d_final_state,
                     mamba2_rows d_q, mamba2_rows d_k, mamba2_rows d_v,
                     mamba2_rows d_g, mamba2_rows d_beta,
                     float* d_initial_state, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * One token of each of `batch` sequences: the tensors of the rule without a
 * token axis (batch_stride; row_stride is not used).  new_state may be `state`
 * itself; any other overlap is refused (MAMBA2_SCAN_EOVERLAP).
 */
int mamba2_delta_step(int batch, mamba2_delta_dims dims, mamba2_rows q,
                      mamba2_rows k, mamba2_rows v, mamba2_rows g,
                      mamba2_rows beta, const float* state, mamba2_rows y,
                      float* new_state, void* stream);

/* ------------------------------------------------------------------------
 * Group norm with an activation, channels last.  For one token and one group
 * of `width` neighbouring channels (channels = groups * width):
 *   h = x                        (MAMBA2_NORM_GATE_FIRST: x silu(gate))
 *   n = (h - mean) / sqrt(mean((h - mean)^2) + eps)
 *   o = n weight + bias
 *   y = o                        (MAMBA2_NORM_SILU: silu(o),
 *                                 MAMBA2_NORM_GATED: o silu(gate))
 * with mean the group's mean (centered), or 0.  silu(v) = v / (1 + e^-v).
 * The statistics are of one token's channels: no token sees another.  They are
 * formed in fp32: the sum of a group's (h - mean)^2 stays within its range.
 *   weight, bias: fp32, [channels], or [width] for all groups (shared), or
 *   NULL (1, 0); a bias needs a weight.
 *   1 <= groups <= 65535, 1 <= width <= 16384, channels <= 2^22; eps > 0.
 *   Pointers are aligned to their elements; rows that are 16-byte aligned with
 *   width * size a multiple of 16 take wide loads.
 *   seqs.offsets: only rows offsets[0] .. offsets[batch] - 1 are read and
 *   written; where the sequences between them end makes no difference.
 */
#define MAMBA2_NORM_PLAIN      0
#define MAMBA2_NORM_SILU       1
#define MAMBA2_NORM_GATED      2
#define MAMBA2_NORM_GATE_FIRST 3
typedef struct {
  int type;      /* of x, gate, y and their gradients                       */
  int groups;
  int width;     /* channels of a group                                     */
  int form;      /* MAMBA2_NORM_*                                           */
  int centered;
  int shared;    /* weight and bias are [width]                             */
  float eps;
} mamba2_norm_dims;

/* gate.data may be NULL for the forms without one. */
int mamba2_norm_fwd(mamba2_seqs seqs, mamba2_norm_dims dims, mamba2_rows x,
                    const float* weight, const float* bias, mamba2_rows gate,
                    mamba2_rows y, void* stream);

/* Bytes of mamba2_norm_bwd's workspace (partial sums of the parameters'
 * gradients); 0 for dimensions that are refused. */
size_t mamba2_norm_bwd_workspace_bytes(mamba2_seqs seqs, mamba2_norm_dims dims);

/*
 * Gradients for given dL/dy: d_x, d_gate (their data may be NULL; d_gate only
 * with a gate), d_weight, d_bias (NULL, or given with the parameter), not all
 * NULL unless there are no rows.  The statistics are recomputed from x.
 * workspace: 16-byte aligned, needed when d_weight or d_bias is.
 */
int mamba2_norm_bwd(mamba2_seqs seqs, mamba2_norm_dims dims, mamba2_rows x,
                    const float* weight, const float* bias, mamba2_rows gate,
                    mamba2_rows d_y, mamba2_rows d_x, float* d_weight,
                    float* d_bias, mamba2_rows d_gate, void* workspace,
                    size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_DELTA_H */
