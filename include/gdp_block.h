/*
 * gdp_block.h -- C ABI of the operators around a recurrence in a block of a recurrent language model, in
 * the same library (libgdp_gb300.so):
 *
 *   - the short causal convolution in front of a recurrence: packed sequences, its backward pass, and the
 *     one-token step of serving;
 *   - the selective state space scan, a recurrence of S values per channel whose step size, input and readout
 *     vectors depend on the token: the same three;
 *   - the residual norm: the norm behind one block, its gate and scale, the residual sum and the norm before
 *     the next block in one pass, and its backward pass.
 *
 * Conventions are those of gdp_layer.h: caller-owned device pointers, no allocation, no synchronisation, all
 * work enqueued on `stream` in order (graph-capturable), a host-side argument error returns a non-zero
 * gdp_status before any launch with the reason in gdp_last_error(), and GDP_DEV_ERR_* bits are OR-ed into
 * *device_status for what only the device can see.  Strides are in elements; the innermost dimension is
 * contiguous.  T is below 2^31.  Any alignment of the elements' own size is served; 16-byte aligned bases and strides
 * take the fast paths.  Outputs must not overlap inputs or one another unless said: of the tensors of T rows, an overlap
 * is GDP_ERR_ALIAS (the gaps between a strided tensor's rows are not its own).  Results do not depend on scheduling: every value
 * is formed by the same operations in the same order.
 *
 * Packed sequences and state modes are those of gdp_linear_recurrence: cu_seqlens that do not ascend from 0 to
 * at most T set GDP_DEV_ERR_CU_SEQLENS (outputs then undefined, nothing outside the buffers touched; with N = 0 every row is
 * padding and they are not read); an empty
 * sequence's final state is its incoming state; output rows at or past cu_seqlens[N] are not written, or with
 * zero_padding written as zeros; the cache `state` is read and written in place at state_indices[i] (-1: start
 * from zero, write nothing; any other value outside [0, num_slots) sets GDP_DEV_ERR_SLOT and is treated as -1; no slot
 * twice), otherwise initial_state (or NULL: zero) is read and output_state (or NULL) written; the two may be the
 * same buffer exactly, a partial overlap is GDP_ERR_ALIAS.
 */
#ifndef GDP_BLOCK_H
#define GDP_BLOCK_H

#include "gdp_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gdp_short_convolution: for every packed sequence and channel c, with W = width taps (2 to 4),
 *
 *     p_t = bias + sum_{j < W} weight[c][j] x_{t - W + 1 + j},   y_t = p_t (GDP_ACT_NONE) or p_t sigmoid(p_t) (GDP_ACT_SILU).
 *
 * Inputs before a sequence's first token come from its incoming state, the W - 1 inputs before it, oldest
 * first: [W - 1, C] per sequence or slot, contiguous, of x's type (states are inputs as they were, so nothing
 * is rounded).  The final state is the last W - 1 inputs, incoming ones among them where the sequence is shorter.
 *
 * gdp_short_convolution_decode: one token per sequence (T == N, token i belongs to sequence i); cu_seqlens is
 * ignored.
 */
typedef struct gdp_conv_args {
  const void *x; /* [T, C], rows x_stride_t apart */
  int64_t x_stride_t;
  const float *weight; /* [C, W] */
  const float *bias;   /* [C] or NULL */
  void *output;        /* [T, C], contiguous, dtype */
  const void *cu_seqlens; /* [N + 1] int32, or int64 when cu_seqlens_int64 != 0 */
  int64_t T, N, C, width;
  const void *initial_state; /* [N, W - 1, C], dtype */
  void *output_state;
  void *state; /* [num_slots, W - 1, C] */
  const int32_t *state_indices;
  int64_t num_slots;
  uint32_t *device_status; /* optional */
  int cu_seqlens_int64;
  int dtype; /* type of x, output and the states: GDP_DTYPE_BF16, _F16 or _F32 */
  int activation;
  int zero_padding;
} gdp_conv_args;

gdp_status gdp_short_convolution(const gdp_conv_args *args, void *stream);
gdp_status gdp_short_convolution_decode(const gdp_conv_args *args, void *stream);

/*
 * gdp_short_convolution_backward: for dL/dy = d_output and dL/dfinal = d_final_state (or NULL: zero), with
 * dp = d_output act'(p),
 *
 *     dx_t = sum_j weight[c][j] dp_{t + W - 1 - j} (+ d_final_state),  d_weight[c][j] = sum_t dp_t x_{t - W + 1 + j},
 *     d_bias = sum_t dp_t,  d_initial_state likewise as dx.
 *
 * The dense state mode only.  dx [T, C] contiguous (rows at or past cu_seqlens[N] are zeros); d_weight, d_bias
 * fp32 (d_bias NULL without a bias); d_initial_state in dtype or NULL.
 */
typedef struct gdp_conv_backward_args {
  const void *x;
  int64_t x_stride_t;
  const float *weight, *bias;
  const void *d_output; /* [T, C] */
  int64_t d_output_stride_t;
  const void *cu_seqlens;
  int64_t T, N, C, width;
  const void *initial_state; /* [N, W - 1, C] or NULL */
  const void *d_final_state; /* [N, W - 1, C] or NULL */
  void *dx;
  float *d_weight, *d_bias;
  void *d_initial_state;
  void *workspace; /* >= gdp_conv_workspace_bytes(T, C, width), 256-byte aligned */
  size_t workspace_bytes;
  uint32_t *device_status;
  int cu_seqlens_int64;
  int dtype;
  int activation;
} gdp_conv_backward_args;

gdp_status gdp_short_convolution_backward(const gdp_conv_backward_args *args, void *stream);
size_t gdp_conv_workspace_bytes(int64_t T, int64_t C, int64_t width); /* 0 for an invalid shape */

/*
 * gdp_selective_scan: for every packed sequence, channel c and state s < S (S up to 64), with
 * e_t = softplus(dt_t + dt_bias) (or dt_t + dt_bias without dt_softplus),
 *
 *     h_t[c][s] = exp(e_t A[c][s]) h_{t-1}[c][s] + e_t x_t[c] B_t[s],
 *     y_t[c]    = sum_s C_t[s] h_t[c][s] + D[c] x_t[c],   times z_t sigmoid(z_t) when z is given.
 *
 * B and C are shared by the C / G consecutive channels of a group (C S up to 33 million, or fewer for groups of few
 * channels, and N times that below 2^40: GDP_ERR_UNSUPPORTED beyond).  States are fp32 [C, S] per sequence or
 * slot, contiguous.  Sums and states are fp32; y is rounded once.
 *
 * chunk_states (optional, what the backward pass reads): the state entering every chunk of GDP_SCAN_CHUNK tokens
 * of every sequence; chunk j of sequence i is row cu_seqlens[i] / GDP_SCAN_CHUNK + i + j of
 * gdp_scan_chunk_rows(T, N) rows [C, S].  Rows that no chunk has are not written.
 *
 * gdp_selective_scan_decode: one token per sequence (T == N); cu_seqlens and chunk_states are ignored.
 */
#define GDP_SCAN_CHUNK 16
typedef struct gdp_scan_args {
  const void *x; /* [T, C], x_dtype */
  int64_t x_stride_t;
  const void *dt; /* [T, C], dt_dtype */
  int64_t dt_stride_t;
  const float *A;         /* [C, S] */
  const void *B, *C_in;   /* [T, G, S], x_dtype; rows and groups at their strides */
  int64_t B_stride_t, B_stride_g, C_stride_t, C_stride_g;
  const float *D;       /* [C] or NULL */
  const void *z;        /* [T, C], x_dtype, or NULL */
  int64_t z_stride_t;
  const float *dt_bias; /* [C] or NULL */
  void *output;         /* [T, C], contiguous, x_dtype */
  const void *cu_seqlens;
  int64_t T, N, C, S, G;
  const float *initial_state; /* [N, C, S] */
  float *output_state;
  float *state; /* [num_slots, C, S] */
  const int32_t *state_indices;
  int64_t num_slots;
  float *chunk_states;
  void *workspace; /* >= gdp_scan_forward_workspace_bytes(T, N, C, S, G), 256-byte aligned; NULL where that is 0 */
  size_t workspace_bytes;
  uint32_t *device_status;
  int cu_seqlens_int64;
  int x_dtype;  /* GDP_DTYPE_BF16, _F16 or _F32 */
  int dt_dtype; /* x_dtype or GDP_DTYPE_F32 */
  int dt_softplus;
  int zero_padding;
} gdp_scan_args;

gdp_status gdp_selective_scan(const gdp_scan_args *args, void *stream);
gdp_status gdp_selective_scan_decode(const gdp_scan_args *args, void *stream);
int64_t gdp_scan_chunk_rows(int64_t T, int64_t N);
/* Few sequences of few channels run in pieces side by side, whose states are joined through this workspace (0: none
   is needed; decode needs none). */
size_t gdp_scan_forward_workspace_bytes(int64_t T, int64_t N, int64_t C, int64_t S, int64_t G);

/*
 * gdp_selective_scan_backward: gradients for dL/dy = d_output and dL/dfinal = d_final_state (or NULL), from
 * the inputs and the chunk_states that the forward call wrote.  With dy = d_output (times silu(z)),
 *
 *     H_t = C_t dy_t + exp(e_{t+1} A) H_{t+1} (at a sequence's last token: C_t dy_t + d_final_state),
 *     u_t = sum_s H_t B_t,  v_t = sum_s H_t exp(e_t A) h_{t-1} A,
 *     dx = u e + dy D,  d(e) = v + u x,  ddt = d(e) sigmoid(dt + dt_bias) (or d(e)),
 *     dB_t = sum_c H_t e_t x_t,  dC_t = sum_c dy_t h_t  (over a group's channels),
 *     dA = sum_t H_t exp(e_t A) h_{t-1} e_t,  dD = sum_t dy_t x_t,  ddt_bias = sum_t ddt,
 *     dz = d_output y' silu'(z) with y' the ungated readout,  d_initial_state = exp(e_0 A) H_0.
 *
 * dx, dz [T, C] x_dtype; ddt dt_dtype; dB, dC [T, G, S] x_dtype, all contiguous; their rows at or past
 * cu_seqlens[N] are zeros.  dA, dD (NULL without D), ddt_bias (NULL without it) fp32.  d_initial_state
 * [N, C, S] or NULL.  The sums over rows and channels run in a fixed order.
 */
typedef struct gdp_scan_backward_args {
  const void *x;
  int64_t x_stride_t;
  const void *dt;
  int64_t dt_stride_t;
  const float *A;
  const void *B, *C_in;
  int64_t B_stride_t, B_stride_g, C_stride_t, C_stride_g;
  const float *D;
  const void *z;
  int64_t z_stride_t;
  const float *dt_bias;
  const void *d_output; /* [T, C], x_dtype */
  int64_t d_output_stride_t;
  const void *cu_seqlens;
  int64_t T, N, C, S, G;
  const float *chunk_states;
  const float *d_final_state; /* [N, C, S] or NULL */
  void *dx, *ddt;
  float *dA;
  void *dB, *dC;
  float *dD;
  void *dz;
  float *ddt_bias;
  float *d_initial_state;
  void *workspace; /* >= gdp_scan_workspace_bytes(T, N, C, S, G), 256-byte aligned */
  size_t workspace_bytes;
  uint32_t *device_status;
  int cu_seqlens_int64;
  int x_dtype, dt_dtype;
  int dt_softplus;
} gdp_scan_backward_args;

gdp_status gdp_selective_scan_backward(const gdp_scan_backward_args *args, void *stream);
size_t gdp_scan_workspace_bytes(int64_t T, int64_t N, int64_t C, int64_t S, int64_t G);

/*
 * gdp_residual_norm: for every token, over its C channels (C up to 8192, row strides below 2^31),
 *
 *     m = block / sqrt(mean(block^2) + eps) post_weight   (m = block without post_weight),
 *     r = residual + scale act(gate) m,   y = r / sqrt(mean(r^2) + eps) weight.
 *
 * act: GDP_ACT_NONE (the gate as it is), _SILU or _SIGMOID; without a gate the factor is one.  weight,
 * post_weight and scale: fp32 [C], the last two optional.  r is kept in fp32 until it is written (in
 * residual_dtype: dtype or fp32); y is formed from the unrounded r.  residual_out may be the residual's
 * own buffer exactly (contiguous rows); a partial overlap is GDP_ERR_ALIAS.
 */
typedef struct gdp_residual_norm_args {
  const void *residual; /* [T, C], residual_dtype */
  int64_t residual_stride_t;
  const void *block; /* [T, C], dtype */
  int64_t block_stride_t;
  const void *gate; /* [T, C], dtype, or NULL */
  int64_t gate_stride_t;
  const float *weight, *post_weight, *scale;
  void *y;            /* [T, C], contiguous, dtype */
  void *residual_out; /* [T, C], contiguous, residual_dtype */
  int64_t T, C;
  float eps;
  int dtype, residual_dtype, activation;
} gdp_residual_norm_args;

gdp_status gdp_residual_norm(const gdp_residual_norm_args *args, void *stream);

/*
 * gdp_residual_norm_backward: gradients for dL/dy = d_y and dL/dr = d_residual_out (or NULL: zero), from the
 * forward's residual_out (as it was stored), block and gate.  d_residual: residual_dtype; d_block, d_gate
 * (NULL without a gate): dtype, contiguous [T, C]; d_weight, d_post_weight, d_scale (NULL where the forward has
 * none): fp32 [C].  d_residual may be d_residual_out's own buffer exactly (contiguous rows).
 */
typedef struct gdp_residual_norm_backward_args {
  const void *d_y; /* [T, C], dtype */
  int64_t d_y_stride_t;
  const void *d_residual_out; /* [T, C], residual_dtype, or NULL */
  int64_t d_residual_out_stride_t;
  const void *residual_out;
  int64_t residual_out_stride_t;
  const void *block;
  int64_t block_stride_t;
  const void *gate;
  int64_t gate_stride_t;
  const float *weight, *post_weight, *scale;
  void *d_residual, *d_block, *d_gate;
  float *d_weight, *d_post_weight, *d_scale;
  void *workspace; /* >= gdp_residual_norm_workspace_bytes(T, C), 256-byte aligned */
  size_t workspace_bytes;
  int64_t T, C;
  float eps;
  int dtype, residual_dtype, activation;
} gdp_residual_norm_backward_args;

gdp_status gdp_residual_norm_backward(const gdp_residual_norm_backward_args *args, void *stream);
size_t gdp_residual_norm_workspace_bytes(int64_t T, int64_t C);

/* Struct sizes as compiled into the library: 0 convolution, 1 its backward, 2 scan, 3 its backward,
   4 residual norm, 5 its backward. */
size_t gdp_block_args_size(int which);

#ifdef __cplusplus
}
#endif
#endif /* GDP_BLOCK_H */
