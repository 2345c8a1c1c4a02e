/*
 * mamba2_layer.h -- C ABI of the selective layer's operators for AMD Instinct
 * MI355X (gfx950): the short causal convolution, the selective state space
 * scan, and gradient clipping.  Part of libmamba2scan.so, beside the temporal
 * scan of mamba2_scan.h, whose status codes it returns.
 *
 * Conventions for every entry point:
 *   - Pointers are device memory owned by the caller (the structs themselves
 *     and the pointer tables of the gradient calls are host memory, read
 *     before the call returns).  The library allocates nothing, keeps no
 *     state between calls and never synchronises: work is enqueued on
 *     `stream` (a hipStream_t; NULL = the null stream) of the current device.
 *   - Every argument check runs before any work is enqueued.  On a nonzero
 *     return nothing has been written, except after MAMBA2_SCAN_EHIP.
 *   - Outputs are overwritten, never accumulated into, and every result is
 *     bitwise reproducible: no atomics, every sum in a fixed order.
 *   - An output may not overlap an input or another output, except where a
 *     call says so.
 *   - Calls whose launch would have 2^32 threads or more are refused
 *     (MAMBA2_SCAN_EBADDIM).  The convolution has 64 (backward: 256) for every 8
 *     to 64 tokens of a sequence and 64 channels (wide accesses: 256 or 512),
 *     the scan up to 256 for every sequence and head and its backward 512 for
 *     every 64 tokens of a sequence and group.
 *   - Calls on different streams, and replays of different captured graphs,
 *     may run concurrently if their outputs and workspaces do not overlap.
 *   - A call may be captured into a graph; the addresses it was given, the
 *     workspace's among them, then belong to the graph.
 *
 * Types: activations are fp32 or bf16 (MAMBA2_F32, MAMBA2_BF16); weights,
 * their gradients and the scan's states are fp32.  bf16 is storage: products
 * accumulate in fp32, and an operand that the call itself computes goes into
 * them with 16 bits or more.
 */
#ifndef MAMBA2_LAYER_H
#define MAMBA2_LAYER_H

#include "mamba2_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A status beside those of mamba2_scan.h, and every status in this header's terms. */
#define MAMBA2_SCAN_EOVERLAP     -8 /* tensors that must be apart overlap     */
const char* mamba2_layer_strerror(int status);

#define MAMBA2_F32  0
#define MAMBA2_BF16 1

/*
 * The sequences of a call.  Dense (offsets NULL): `batch` sequences of
 * `length` tokens each.  Packed: one run of `length` rows in which sequence s
 * has the rows offsets[s] .. offsets[s + 1] - 1 (offsets[batch + 1], int32, on
 * the device, nondecreasing, within 0 .. length).  Sequences may be empty.
 * Rows before the first and behind the last sequence are neither read nor
 * written.  Offsets outside that order are clamped into it: results are then
 * unspecified, but no access leaves the tensors.
 * 1 <= batch, 0 <= length, batch * length <= 2^31 - 65536.
 */
typedef struct {
  int batch;
  int length;
  const int* offsets;
} mamba2_seqs;

/*
 * A token-major tensor: element e of token t of sequence s is at
 * data + s * batch_stride + t * row_stride + e, strides in elements (with
 * offsets: row r at data + r * row_stride).  So a tensor may be a slice of a
 * wider one.  Strides are not negative, and rows do not overlap.  Where there
 * is one row, or one sequence (or offsets), row_stride or batch_stride is not
 * used and may be anything.
 */
typedef struct {
  void* data;
  long long batch_stride;
  long long row_stride;
} mamba2_rows;

/* ------------------------------------------------------------------------
 * Short causal depthwise convolution.  For channel c of a sequence
 *   y_t = f(bias + sum_{k < taps} weight[c][k] x_{t - taps + 1 + k}),
 * f the identity or SiLU (v / (1 + e^-v)); x before the sequence's start comes
 * from initial_state [batch][taps - 1][channels] (oldest first, x's type), or
 * is 0 when that is NULL.  final_state (the same layout; NULL skips it) gets
 * the last taps - 1 inputs, which start the next piece of the sequence.
 *   1 <= channels <= 2^22, row strides up to 2^22 elements, taps 2, 3 or 4; weight [channels][taps], bias [channels]
 *   or NULL.  Pointers are aligned to their elements; rows that are 16-byte
 *   aligned with channels * size a multiple of 16 take wide loads.
 */
int mamba2_conv_fwd(int type, mamba2_seqs seqs, int channels, int taps, int silu,
                    mamba2_rows x, const float* weight, const float* bias,
                    const void* initial_state, mamba2_rows y, void* final_state,
                    void* stream);

/* Bytes of mamba2_conv_bwd's workspace (partial sums of the weights'
 * gradients); 0 for dimensions that are refused. */
size_t mamba2_conv_bwd_workspace_bytes(mamba2_seqs seqs, int channels, int taps);

/*
 * Gradients for given dL/dy and, when not NULL, dL/dfinal_state: d_x (its
 * data may be NULL), d_weight, d_bias, d_initial_state (each may be NULL, not
 * all).  The pre-activation is recomputed from x.  workspace: 16-byte
 * aligned, needed when d_weight or d_bias is.
 */
int mamba2_conv_bwd(int type, mamba2_seqs seqs, int channels, int taps, int silu,
                    mamba2_rows x, const float* weight, const float* bias,
                    const void* initial_state, mamba2_rows d_y,
                    const void* d_final_state, mamba2_rows d_x, float* d_weight,
                    float* d_bias, void* d_initial_state, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * One token of each of `batch` <= 65535 sequences: x and y [batch][channels]
 * (their batch_stride; row_stride is not used), state [batch][taps - 1][channels].
 * new_state gets the state moved on by the token; it may be `state` itself.
 * Any other overlap is refused (MAMBA2_SCAN_EOVERLAP).
 */
int mamba2_conv_step(int type, int batch, int channels, int taps, int silu,
                     mamba2_rows x, const float* weight, const float* bias,
                     const void* state, mamba2_rows y, void* new_state,
                     void* stream);

/* ------------------------------------------------------------------------
 * Selective state space scan.  Per sequence and head h, with the state
 * S [states][width] (fp32), g = h / (heads / groups) and
 * d_t = softplus(dt_t + dt_bias) (softplus only if dims.softplus; dt_bias may
 * be NULL):
 *   S_t = exp(d_t A_h) S_{t-1} + d_t B_t[g] x_t[h]^T
 *   y_t[h] = S_t^T C_t[g] + D_h x_t[h]             (D may be NULL)
 *   x, y [heads][width], dt [heads], B, C [groups][states] per token;
 *   A, D, dt_bias [heads]; states' layout [batch][heads][states][width].
 * S_0 = initial_state (NULL: 0); final_state (NULL: skipped) gets the state
 * after the last token, and initial_state itself for an empty sequence.
 * A token whose d_t is 0 (dt = -inf under softplus) leaves the state as it
 * was; so a padded batch marks its padding, x, B and C there being finite.
 *   1 <= groups, heads a multiple of groups, at most 65535, as batch is;
 *   width and states multiples of 8, 8 .. 128.  x, B, C, y and the states are
 *   16-byte aligned, with row and batch strides that are multiples of 8
 *   elements; dt has any stride.  Row strides are at most 2^29 / 65 elements.
 *   A value of x, B, C, dt or d_y that is not finite may reach every token of
 * its own sequence from the start of its step of 64 tokens on (gradients: up
 * to the end of it and before), but no other sequence; an infinity may come out
 * as a NaN.  A NaN in A (D, dt_bias)
 * reaches every token of its head (groups share d_B and d_C).  A = -inf: every
 * token but those whose d_t is 0 forgets the state.
 *   A <= 0 is meant; growing states (A > 0) are computed as long as the decay
 *   over 128 tokens stays finite.
 */
typedef struct {
  int type;     /* of x, B, C, y and their gradients                        */
  int dt_type;  /* of dt and its gradient                                   */
  int heads;
  int width;    /* elements of a head (P)                                   */
  int groups;   /* heads / groups neighbouring heads share one B and C      */
  int states;   /* elements of B and C (N)                                  */
  int softplus;
} mamba2_ssm_dims;

/* Bytes of the forward's workspace; 0 when none is needed, and for
 * dimensions that are refused. */
size_t mamba2_ssm_fwd_workspace_bytes(mamba2_seqs seqs, mamba2_ssm_dims dims);

int mamba2_ssm_fwd(mamba2_seqs seqs, mamba2_ssm_dims dims, mamba2_rows x,
                   mamba2_rows dt, const float* A, mamba2_rows B, mamba2_rows C,
                   const float* D, const float* dt_bias,
                   const float* initial_state, mamba2_rows y,
                   float* final_state, void* workspace, size_t workspace_bytes,
                   void* stream);

/* Bytes of the backward's workspace: the states at the chunks' borders, both
 * ways, and partial sums; 0 for dimensions that are refused. */
size_t mamba2_ssm_bwd_workspace_bytes(mamba2_seqs seqs, mamba2_ssm_dims dims);

/*
 * Gradients for given dL/dy and, when not NULL, dL/dfinal_state.  The states
 * are recomputed from the inputs.  d_x, d_dt, d_A, d_B, d_C are required;
 * d_D (required D), d_dt_bias and d_initial_state may be NULL.  The tensors
 * that the forward was given are given again.
 */
int mamba2_ssm_bwd(mamba2_seqs seqs, mamba2_ssm_dims dims, mamba2_rows x,
                   mamba2_rows dt, const float* A, mamba2_rows B, mamba2_rows C,
                   const float* D, const float* dt_bias,
                   const float* initial_state, mamba2_rows d_y,
                   const float* d_final_state, mamba2_rows d_x,
                   mamba2_rows d_dt, float* d_A, mamba2_rows d_B,
                   mamba2_rows d_C, float* d_D, float* d_dt_bias,
                   float* d_initial_state, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * One token of each of `batch` sequences: the tensors of the scan without a
 * token axis (batch_stride; row_stride is not used).  new_state may be
 * `state` itself; any other overlap is refused (MAMBA2_SCAN_EOVERLAP).
 */
int mamba2_ssm_step(int batch, mamba2_ssm_dims dims, mamba2_rows x,
                    mamba2_rows dt, const float* A, mamba2_rows B,
                    mamba2_rows C, const float* D, const float* dt_bias,
                    const float* state, mamba2_rows y, float* new_state,
                    void* stream);

/* ------------------------------------------------------------------------
 * The global 2-norm of many gradient tensors, and clipping by it.
 * `grads` are count contiguous tensors (a host table), aligned to their
 * elements; count >= 1, numel >= 0, the sum of numel < 2^46.  Squares are
 * summed in 64 bits.
 */
typedef struct {
  const void* grad;
  void* out;        /* mamba2_clip_grads; may be grad itself                */
  long long numel;
  int type;         /* MAMBA2_F32 or MAMBA2_BF16                            */
} mamba2_grad;

/* Bytes of the workspace of both calls; 0 for tables that are refused. */
size_t mamba2_grad_workspace_bytes(const mamba2_grad* grads, int count);

/* *norm = sqrt(sum of squares of every element), fp32.  The gradients may
 * overlap one another, but not norm or the workspace (MAMBA2_SCAN_EOVERLAP). */
int mamba2_grad_norm(const mamba2_grad* grads, int count, float* norm,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * *norm as above, and out = grad * min(1, max_norm / (norm + 1e-6)) for every
 * tensor.  max_norm >= 0 (infinity clips nothing but a NaN).  A NaN among the
 * gradients makes every output NaN; an infinite one makes the factor 0.  The tensors
 * may not overlap one another, norm or the workspace; out overlaps grad only
 * by being it (MAMBA2_SCAN_EOVERLAP otherwise).
 */
int mamba2_clip_grads(const mamba2_grad* grads, int count, float max_norm,
                      float* norm, void* workspace, size_t workspace_bytes,
                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_LAYER_H */
