/*
 * gdp_layer.h -- C ABI of the operators that stand beside the Gated DeltaProduct recurrence
 * (gdp_prefill.h) in a recurrent language model, in the same library (libgdp_gb300.so):
 *
 *   - the gated linear recurrence, a recurrent layer whose state is one value per channel:
 *     packed sequences, its backward pass, and the one-token step of serving;
 *   - the grouped norm with an activated gate, the output stage behind either recurrence
 *     (groups = the heads of a token, channels last), and its backward pass;
 *   - 8-bit activation checkpoints: the norm's forward pass writes them beside its output, and
 *     both backward passes read them in place of the 16-bit activations.
 *
 * Conventions are those of gdp_prefill.h: caller-owned device pointers, no allocation, no
 * synchronisation, all work enqueued on `stream` in order (graph-capturable), a host-side argument
 * error returns a non-zero gdp_status before any launch with the reason in gdp_last_error(), and
 * GDP_DEV_ERR_* bits are OR-ed into *device_status for what only the device can see.  Strides are in
 * elements; the innermost dimension is contiguous.  Any alignment of the elements' own size is
 * served; 16-byte aligned bases and strides take the fast paths.
 */
#ifndef GDP_LAYER_H
#define GDP_LAYER_H

#include "gdp_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the gate value g gives the decay a_t and the recurrence's input b_t. */
typedef enum gdp_gate {
  GDP_GATE_LOG = 0,    /* a = exp(g),     b = x            (natural-log decay, as gdp_prefill's g) */
  GDP_GATE_ALPHA = 1,  /* a = g,          b = x            (the decay itself) */
  GDP_GATE_SIGMOID = 2 /* a = sigmoid(g), b = (1 - a) x    (a convex combination of state and input) */
} gdp_gate;

/*
 * gdp_linear_recurrence: for every packed sequence and channel c,
 *
 *     h_t = a_t h_{t-1} + b_t,   h_{-1} = the incoming state,   final state = h of the last token.
 *
 * An empty sequence's final state is its incoming state.  Rows at or past cu_seqlens[N] (a padded
 * batch's) are not written, or with zero_padding written as zeros; they are not read into any result.
 * cu_seqlens that do not ascend from 0 to at most T set GDP_DEV_ERR_CU_SEQLENS; the
 * outputs are then undefined (nothing outside the buffers is touched).  A sequence's values never
 * depend on another sequence's, infinities and NaN included.  Results do not depend on scheduling:
 * every value is formed by the same operations in the same order.  Gates may be of any size: decays above
 * one, of zero, and any run of them; only the states, and the states that a run of tokens makes from zero,
 * have to stay within fp32.  (Values below 2^-125 may come out as zero; a sigmoid gate is never closed
 * further than 2^-125.)
 *
 * gdp_linear_recurrence_decode: one token per sequence (T == N, token i belongs to sequence i);
 * cu_seqlens is ignored.
 *
 * State modes as for the prefill: the cache `state` [num_slots, C] is read and written in place at
 * state_indices[i] (-1: start from zero, write nothing; any other value outside [0, num_slots) sets
 * GDP_DEV_ERR_SLOT and is treated as -1); otherwise initial_state [N, C] (or NULL: zero) is read and
 * output_state [N, C] (or NULL) written; the two may be the same buffer exactly, a partial overlap is
 * GDP_ERR_ALIAS.  States are fp32, contiguous.  output must not overlap an input.
 */
typedef struct gdp_recurrence_args {
  const void *x;  /* [T, C], rows x_stride_t apart; x_dtype */
  int64_t x_stride_t;
  const void *g;  /* [T, C], rows g_stride_t apart; g_dtype */
  int64_t g_stride_t;
  void *output;   /* h [T, C], contiguous, x_dtype */
  const void *cu_seqlens; /* [N + 1] int32, or int64 when cu_seqlens_int64 != 0 */
  int64_t T, N, C;
  const float *initial_state;
  float *output_state;
  float *state;
  const int32_t *state_indices;
  int64_t num_slots;
  uint32_t *device_status; /* optional */
  int cu_seqlens_int64;
  int x_dtype; /* GDP_DTYPE_BF16, _F16 or _F32 */
  int g_dtype; /* x_dtype or GDP_DTYPE_F32 */
  int gate;    /* gdp_gate */
  int zero_padding; /* nonzero: output rows at or past cu_seqlens[N] are written as zeros */
} gdp_recurrence_args;

gdp_status gdp_linear_recurrence(const gdp_recurrence_args *args, void *stream);
gdp_status gdp_linear_recurrence_decode(const gdp_recurrence_args *args, void *stream);

/*
 * gdp_linear_recurrence_backward: for a loss with dL/dh = d_output and dL/dfinal = d_final_state,
 *
 *     D_t = d_output_t + a_{t+1} D_{t+1}   (at a sequence's last token: + d_final_state)
 *     dx = D (times 1 - a for the sigmoid gate),   dL/da_t = D_t (h_{t-1} [- x_t]),
 *     dg = dL/da times da/dg,   d_initial_state = a_0 D_0.
 *
 * h is the forward's output, either as it was written (h [T, C], d_output's type) or as an 8-bit
 * checkpoint (h_codes [T, C] int8 contiguous with h_scales, whose blocks are laid out as
 * gdp_group_norm writes them for rows of h_group channels: C a multiple of h_group).  Exactly one of h
 * and h_codes is given.  x is needed for the sigmoid gate only.  The dense state mode only.  dx takes
 * x_dtype, dg g_dtype, both contiguous [T, C]; d_initial_state [N, C] fp32 or NULL (an empty sequence's
 * is its d_final_state).  dx and dg rows at or past cu_seqlens[N] are written as zeros, so that sums over
 * all rows are those over the sequences'.
 */
typedef struct gdp_recurrence_backward_args {
  const void *g;
  int64_t g_stride_t;
  const void *x; /* GDP_GATE_SIGMOID only */
  int64_t x_stride_t;
  const void *h;
  int64_t h_stride_t;
  const int8_t *h_codes;
  const float *h_scales;
  int64_t h_group;
  const void *d_output; /* [T, C], x_dtype */
  int64_t d_output_stride_t;
  const void *cu_seqlens;
  int64_t T, N, C;
  const float *initial_state; /* [N, C] or NULL */
  const float *d_final_state; /* [N, C] or NULL (zero) */
  void *dx, *dg;
  float *d_initial_state;
  uint32_t *device_status;
  int cu_seqlens_int64;
  int x_dtype; /* type of x, h, d_output and dx */
  int g_dtype; /* type of g and dg: x_dtype or GDP_DTYPE_F32 */
  int gate;
} gdp_recurrence_backward_args;

gdp_status gdp_linear_recurrence_backward(const gdp_recurrence_backward_args *args, void *stream);

/*
 * gdp_arm_recurrence_wait_test: a test of the failure path, as gdp_arm_wait_expiry_test is for the
 * prefill.  The waits of the calling thread's next gdp_linear_recurrence or _backward call give up after
 * limit_ns (1e5 .. 1e9 ns), and the first tile's contribution to the chain is withheld, so that one of
 * them runs out: GDP_DEV_ERR_TIMEOUT in *device_status, outputs undefined, later calls unaffected.
 * GDP_ERR_INVALID_ARG for a limit outside the range.
 */
gdp_status gdp_arm_recurrence_wait_test(uint64_t limit_ns);

/* What the normed value is multiplied with (z given) or passed through (z NULL). */
typedef enum gdp_activation {
  GDP_ACT_NONE = 0,    /* y = u */
  GDP_ACT_SILU = 1,    /* y = u z sigmoid(z); without z: y = u sigmoid(u) */
  GDP_ACT_SIGMOID = 2  /* y = u sigmoid(z); z required */
} gdp_activation;

/*
 * gdp_group_norm: for every token t and head h, over its D channels (channels last),
 *
 *     n = (o - m) / sqrt(mean((o - m)^2) + eps),   m = mean(o) when `center`, else 0,
 *     u = n weight (+ bias),   y = u act(z).
 *
 * weight and bias: fp32, [D], or [H, D] when per_head.  1 <= D <= 8192.  Sums are fp32.
 *
 * 8-bit checkpoints (optional): o_codes, z_codes [T, H, D] int8 and o_scales, z_scales
 * [T, H, ceil(D / 128)] fp32, written in the same pass.  Each row is cut into blocks of 128 channels
 * (the last one shorter); k = 127 / amax of the block cut to four significant bits,
 * code = round-to-even(value k), scale = 1 / k, and the code stands for code * scale.  (Four bits, so
 * that value k is exact for 16-bit values and the codes are the same in any arithmetic; of an fp32
 * value the product is rounded to fp32 first.  At most 1/9 of the code range stays unused.)  A block
 * whose amax is below 2^-100 is all zeros with scale 0; a block holding an infinity or a NaN gets
 * scale NaN, so that its values, and what is computed from them, are NaN.  (Where 120 scale would be 2^128,
 * beyond fp32, the scale is the next number below 1 / k: every finite block's values are finite.)  Both of a pair, or neither;
 * z's only with z.
 */
typedef struct gdp_group_norm_args {
  const void *o; /* [T, H, D] */
  int64_t o_stride_t, o_stride_h;
  const void *z; /* [T, H, D] or NULL */
  int64_t z_stride_t, z_stride_h;
  const float *weight, *bias; /* bias may be NULL */
  void *y; /* [T, H, D], contiguous, dtype */
  int8_t *o_codes;
  float *o_scales;
  int8_t *z_codes;
  float *z_scales;
  int64_t T, H, D;
  float eps;
  int dtype; /* type of o, z and y: GDP_DTYPE_BF16, _F16 or _F32 */
  int center, per_head, activation;
} gdp_group_norm_args;

gdp_status gdp_group_norm(const gdp_group_norm_args *args, void *stream);

/*
 * gdp_group_norm_backward: gradients of gdp_group_norm for dL/dy = d_y.  o (and z) are read either as
 * tensors or as the checkpoints the forward pass wrote (o_codes / o_scales, z_codes / z_scales); the
 * statistics are recomputed from what is read.  do, dz: [T, H, D] contiguous in dtype; dweight (and
 * dbias, NULL without a bias): fp32 in weight's shape.  The sums over rows run in a fixed order.
 */
typedef struct gdp_group_norm_backward_args {
  const void *d_y; /* [T, H, D] */
  int64_t d_y_stride_t, d_y_stride_h;
  const void *o;
  int64_t o_stride_t, o_stride_h;
  const void *z;
  int64_t z_stride_t, z_stride_h;
  const int8_t *o_codes;
  const float *o_scales;
  const int8_t *z_codes;
  const float *z_scales;
  const float *weight, *bias;
  void *d_o, *d_z;
  float *d_weight, *d_bias;
  void *workspace; /* >= gdp_group_norm_workspace_bytes(T, H, D, per_head), 256-byte aligned */
  size_t workspace_bytes;
  int64_t T, H, D;
  float eps;
  int dtype;
  int center, per_head, activation;
} gdp_group_norm_backward_args;

gdp_status gdp_group_norm_backward(const gdp_group_norm_backward_args *args, void *stream);

/* Workspace bytes of gdp_group_norm_backward (0 for an invalid shape). */
size_t gdp_group_norm_workspace_bytes(int64_t T, int64_t H, int64_t D, int per_head);

/* Struct sizes as compiled into the library (lets a binding check its layouts): 0 recurrence,
   1 recurrence backward, 2 group norm, 3 group norm backward. */
size_t gdp_layer_args_size(int which);

#ifdef __cplusplus
}
#endif
#endif /* GDP_LAYER_H */
