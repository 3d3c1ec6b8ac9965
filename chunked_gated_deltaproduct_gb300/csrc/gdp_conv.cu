// gdp_conv.cu -- the short causal convolution's C entries and argument checks (gdp_block.h), and the column sums that
// the backward passes of gdp_block.h share.
#include "gdp_conv.cuh"

namespace gdp {
namespace layer {
namespace {

// 32 columns per CTA, each warp a stride of the parts, then the warps' sums in turn.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) gdp_column_sums_kernel(const ColumnSums s) {
  __shared__ float sums[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (col < s.cols) {
#pragma unroll 4
    for (int64_t i = warp; i < s.parts; i += kSumWarps) v += s.from[i * s.cols + col];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || col >= s.cols) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kSumWarps; ++i) v += sums[i][lane];
  int seg = 0;
#pragma unroll
  for (int k = 1; k < 4; ++k)
    if (col >= s.first[k]) seg = k;
  int64_t at = col - s.first[seg];
  if (seg == 0 && s.taps) at = (at % s.width) * s.taps + at / s.width;
  if (s.to[seg]) s.to[seg][at] = v;
}

gdp_status conv_ok(int64_t T, int64_t N, int64_t C, int64_t width, int type, int act, const float *w, const float *b) {
  const gdp_status st = shape_ok(T, N, C);
  if (st != GDP_OK) return st;
  if (!dtype_ok(type)) return fail(GDP_ERR_UNSUPPORTED, "dtype must be GDP_DTYPE_BF16, GDP_DTYPE_F16 or GDP_DTYPE_F32");
  if (width < 2 || width > 4) return fail(GDP_ERR_UNSUPPORTED, "width must be 2, 3 or 4");
  if (act != GDP_ACT_NONE && act != GDP_ACT_SILU) return fail(GDP_ERR_INVALID_ARG, "activation must be GDP_ACT_NONE or GDP_ACT_SILU");
  if (!w) return fail(GDP_ERR_INVALID_ARG, "weight is required");
  if (!aligned(w, 4) || !aligned(b, 4)) return fail(GDP_ERR_INVALID_ARG, "fp32 buffers must be 4-byte aligned");
  return GDP_OK;
}

gdp_status resolve(const gdp_conv_args *a, bool step, ConvProblem *p) {
  set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  gdp_status st = conv_ok(a->T, a->N, a->C, a->width, a->dtype, a->activation, a->weight, a->bias);
  if (st != GDP_OK) return st;
  if (step && a->T != a->N) return fail(GDP_ERR_INVALID_ARG, "decode takes one token per sequence: T == N");
  if ((st = rows_ok(a->x, a->x_stride_t, a->T, a->C, a->dtype, "x")) != GDP_OK) return st;
  if ((st = rows_ok(a->output, a->C, a->T, a->C, a->dtype, "output")) != GDP_OK) return st;
  if (!step && !a->cu_seqlens) return fail(GDP_ERR_INVALID_ARG, "cu_seqlens is required");
  const size_t es = dtype_size(a->dtype);
  if ((st = states_ok(a->initial_state, a->output_state, a->state, a->state_indices, a->num_slots, es,
                      es * (size_t)a->N * (size_t)(a->width - 1) * (size_t)a->C)) != GDP_OK)
    return st;
  if ((st = apart_ok(a->T, {dense(a->output, a->C, a->dtype, "output")}, {rows(a->x, stride_of(a->x_stride_t, a->T, a->C), a->C, a->dtype, "x")})) != GDP_OK)
    return st;
  *p = ConvProblem{};
  p->x = a->x; p->x_st = stride_of(a->x_stride_t, a->T, a->C);
  p->w = a->weight; p->b = a->bias; p->y = a->output;
  p->p = Packed{a->cu_seqlens, a->cu_seqlens_int64 != 0, a->T, a->N, a->device_status};
  p->C = a->C;
  p->s = StateModes{a->initial_state, a->output_state, a->state, a->state_indices, a->num_slots};
  p->act = a->activation;
  p->zero_pad = a->zero_padding != 0;
  p->quad_taps = aligned(a->weight, 16);
  return GDP_OK;
}

// Channels per thread: the widest of 16 bytes, two and one that every tensor's rows allow.
int vec_of(const ConvProblem &p, int type, int most) {
  for (int v = most; v > 1; v = v > 2 ? 2 : 1) {
    const size_t bytes = v * dtype_size(type);
    if (p.C % v == 0 && rows_by(p.x, p.x_st, p.p.T, type, bytes) && rows_by(p.dy, p.dy_st, p.p.T, type, bytes) && aligned(p.y, bytes) &&
        aligned(p.dx, bytes) && aligned(p.s.init, bytes) && aligned(p.s.fin, bytes) && aligned(p.s.cache, bytes) && aligned(p.dfin, bytes) &&
        aligned(p.dinit, bytes))
      return v;
  }
  return 1;
}

}  // namespace

cudaError_t launch_column_sums(const ColumnSums &s, cudaStream_t stream) {
  gdp_column_sums_kernel<<<(unsigned)((s.cols + 31) / 32), 32 * kSumWarps, 0, stream>>>(s);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace gdp

GDP_EXPORT gdp_status gdp_short_convolution(const gdp_conv_args *args, void *stream) {
  using namespace gdp::layer;
  ConvProblem p;
  const gdp_status st = resolve(args, false, &p);
  if (st != GDP_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (p.p.N == 0) return args->zero_padding ? zero_out(p.y, (size_t)(p.p.T * p.C), args->dtype, s) : GDP_OK;
  const int vec = vec_of(p, args->dtype, 16 / dtype_size(args->dtype)), width = (int)args->width, type = args->dtype;
  // A state that is updated in place is still read while rows are worked on: it is written by a second kernel.
  const bool later = p.s.cache || (p.s.fin && p.s.fin == p.s.init), now = p.s.fin && !later;
  cudaError_t e = type == GDP_DTYPE_BF16  ? launch_conv_fwd<__nv_bfloat16>(p, width, vec, now, s)
                  : type == GDP_DTYPE_F16 ? launch_conv_fwd<__half>(p, width, vec, now, s)
                                          : launch_conv_fwd<float>(p, width, vec, now, s);
  if (e == cudaSuccess && later)
    e = type == GDP_DTYPE_BF16  ? launch_conv_states<__nv_bfloat16>(p, width, s)
        : type == GDP_DTYPE_F16 ? launch_conv_states<__half>(p, width, s)
                                : launch_conv_states<float>(p, width, s);
  return cuda_status(e, "short convolution kernel");
}

GDP_EXPORT gdp_status gdp_short_convolution_decode(const gdp_conv_args *args, void *stream) {
  using namespace gdp::layer;
  ConvProblem p;
  const gdp_status st = resolve(args, true, &p);
  if (st != GDP_OK || p.p.N == 0) return st;
  const int width = (int)args->width, type = args->dtype;
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(type == GDP_DTYPE_BF16  ? launch_conv_step<__nv_bfloat16>(p, width, s)
                     : type == GDP_DTYPE_F16 ? launch_conv_step<__half>(p, width, s)
                                             : launch_conv_step<float>(p, width, s),
                     "short convolution step kernel");
}

GDP_EXPORT size_t gdp_conv_workspace_bytes(int64_t T, int64_t C, int64_t width) {
  using namespace gdp::layer;
  if (T < 0 || C < 1 || T > INT32_MAX || C > (1 << 20) || width < 2 || width > 4) return 0;
  int64_t parts = 1;
  for (int64_t v = 1; v <= 4; v *= 2) {
    const int64_t n = conv_parts(T, (C + v - 1) / v, sm_count());
    if (n > parts) parts = n;
  }
  return ((size_t)parts * (size_t)(width + 1) * (size_t)C * 4 + 255) / 256 * 256;
}

GDP_EXPORT gdp_status gdp_short_convolution_backward(const gdp_conv_backward_args *a, void *stream) {
  using namespace gdp::layer;
  gdp::set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  gdp_status st = conv_ok(a->T, a->N, a->C, a->width, a->dtype, a->activation, a->weight, a->bias);
  if (st != GDP_OK) return st;
  if ((st = rows_ok(a->x, a->x_stride_t, a->T, a->C, a->dtype, "x")) != GDP_OK) return st;
  if ((st = rows_ok(a->d_output, a->d_output_stride_t, a->T, a->C, a->dtype, "d_output")) != GDP_OK) return st;
  if ((st = rows_ok(a->dx, a->C, a->T, a->C, a->dtype, "dx")) != GDP_OK) return st;
  if (!a->cu_seqlens) return fail(GDP_ERR_INVALID_ARG, "cu_seqlens is required");
  if (!a->d_weight || (a->bias != nullptr) != (a->d_bias != nullptr))
    return fail(GDP_ERR_INVALID_ARG, "d_weight is required, d_bias goes with bias");
  const size_t es = dtype_size(a->dtype);
  if (!aligned(a->initial_state, es) || !aligned(a->d_final_state, es) || !aligned(a->d_initial_state, es) || !aligned(a->d_weight, 4) ||
      !aligned(a->d_bias, 4))
    return fail(GDP_ERR_INVALID_ARG, "buffers must be aligned to their elements");
  const size_t bytes = es * (size_t)a->N * (size_t)(a->width - 1) * (size_t)a->C;
  if (overlap(a->d_final_state, a->d_initial_state, bytes) || overlap(a->initial_state, a->d_initial_state, bytes))
    return fail(GDP_ERR_ALIAS, "d_initial_state overlaps initial_state or d_final_state");
  if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < gdp_conv_workspace_bytes(a->T, a->C, a->width))
    return fail(GDP_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than gdp_conv_workspace_bytes");
  if ((st = apart_ok(a->T, {dense(a->dx, a->C, a->dtype, "dx")},
                     {rows(a->x, stride_of(a->x_stride_t, a->T, a->C), a->C, a->dtype, "x"),
                      rows(a->d_output, stride_of(a->d_output_stride_t, a->T, a->C), a->C, a->dtype, "d_output")})) != GDP_OK)
    return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (a->N == 0) {  // every row is padding
    if ((st = zero_out(a->dx, (size_t)(a->T * a->C), a->dtype, s)) != GDP_OK) return st;
    if ((st = zero_out(a->d_weight, (size_t)(a->C * a->width), GDP_DTYPE_F32, s)) != GDP_OK) return st;
    return zero_out(a->d_bias, (size_t)a->C, GDP_DTYPE_F32, s);
  }
  ConvProblem p{};
  p.x = a->x; p.x_st = stride_of(a->x_stride_t, a->T, a->C);
  p.w = a->weight; p.b = a->bias;
  p.p = Packed{a->cu_seqlens, a->cu_seqlens_int64 != 0, a->T, a->N, a->device_status};
  p.C = a->C;
  p.s.init = a->initial_state;
  p.act = a->activation; p.quad_taps = aligned(a->weight, 16);
  p.dy = a->d_output; p.dy_st = stride_of(a->d_output_stride_t, a->T, a->C);
  p.dfin = a->d_final_state; p.dx = a->dx; p.dinit = a->d_initial_state;
  p.partial = static_cast<float *>(a->workspace);
  const int width = (int)a->width, vec = vec_of(p, a->dtype, 4);
  cudaError_t e = a->dtype == GDP_DTYPE_BF16  ? launch_conv_bwd<__nv_bfloat16>(p, width, vec, s)
                  : a->dtype == GDP_DTYPE_F16 ? launch_conv_bwd<__half>(p, width, vec, s)
                                              : launch_conv_bwd<float>(p, width, vec, s);
  if (e == cudaSuccess) {
    ColumnSums c{};
    c.from = p.partial; c.parts = p.parts; c.cols = (width + 1) * p.C;
    c.to[0] = a->d_weight; c.to[1] = a->d_bias;
    c.first[1] = width * p.C; c.first[2] = c.first[3] = c.cols;
    c.taps = width; c.width = p.C;
    e = launch_column_sums(c, s);
  }
  return cuda_status(e, "short convolution backward kernels");
}
