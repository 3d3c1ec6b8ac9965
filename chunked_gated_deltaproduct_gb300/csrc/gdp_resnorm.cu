// gdp_resnorm.cu -- the residual norm's C entries and argument checks (gdp_block.h).
#include <initializer_list>

#include "gdp_resnorm.cuh"

namespace gdp {
namespace layer {
namespace {

gdp_status res_ok(int64_t T, int64_t C, float eps, int type, int res_type, int act, const float *w, const float *post, const float *scale) {
  if (T < 0 || C < 1) return fail(GDP_ERR_INVALID_ARG, "T >= 0 and C >= 1 are required");
  if (C > kResMost || T > INT32_MAX) return fail(GDP_ERR_UNSUPPORTED, "C up to 8192, T below 2^31");
  if (!dtype_ok(type)) return fail(GDP_ERR_UNSUPPORTED, "dtype must be GDP_DTYPE_BF16, GDP_DTYPE_F16 or GDP_DTYPE_F32");
  if (res_type != type && res_type != GDP_DTYPE_F32) return fail(GDP_ERR_UNSUPPORTED, "residual_dtype must be dtype or GDP_DTYPE_F32");
  if (!(eps >= 0.f)) return fail(GDP_ERR_INVALID_ARG, "eps must not be negative");
  if (act != GDP_ACT_NONE && act != GDP_ACT_SILU && act != GDP_ACT_SIGMOID)
    return fail(GDP_ERR_INVALID_ARG, "activation must be GDP_ACT_NONE, GDP_ACT_SILU or GDP_ACT_SIGMOID");
  if (!w) return fail(GDP_ERR_INVALID_ARG, "weight is required");
  if (!aligned(w, 4) || !aligned(post, 4) || !aligned(scale, 4)) return fail(GDP_ERR_INVALID_ARG, "fp32 buffers must be 4-byte aligned");
  return GDP_OK;
}
// Row strides that the kernels take (32 bits).
bool short_strides(std::initializer_list<int64_t> strides) {
  for (int64_t s : strides)
    if (s > INT32_MAX) return false;
  return true;
}
// The stream's rows may be replaced: its own buffer exactly, or others.
bool partly(const void *in, int64_t stride, const void *out, int64_t T, int64_t C, int type) {
  return T > 0 && !(in == out && stride == C) && spans_overlap(rows(in, stride, C, type, ""), dense(out, C, type, ""), T);
}

}  // namespace
}  // namespace layer
}  // namespace gdp

GDP_EXPORT gdp_status gdp_residual_norm(const gdp_residual_norm_args *a, void *stream) {
  using namespace gdp::layer;
  gdp::set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  gdp_status st = res_ok(a->T, a->C, a->eps, a->dtype, a->residual_dtype, a->activation, a->weight, a->post_weight, a->scale);
  if (st != GDP_OK) return st;
  if ((st = rows_ok(a->residual, a->residual_stride_t, a->T, a->C, a->residual_dtype, "residual")) != GDP_OK) return st;
  if ((st = rows_ok(a->block, a->block_stride_t, a->T, a->C, a->dtype, "block")) != GDP_OK) return st;
  if (a->gate && (st = rows_ok(a->gate, a->gate_stride_t, a->T, a->C, a->dtype, "gate")) != GDP_OK) return st;
  if ((st = rows_ok(a->y, a->C, a->T, a->C, a->dtype, "y")) != GDP_OK) return st;
  if ((st = rows_ok(a->residual_out, a->C, a->T, a->C, a->residual_dtype, "residual_out")) != GDP_OK) return st;
  ResProblem p{};
  p.res = a->residual; p.block = a->block; p.gate = a->gate;
  p.res_st = stride_of(a->residual_stride_t, a->T, a->C); p.block_st = stride_of(a->block_stride_t, a->T, a->C);
  p.gate_st = stride_of(a->gate_stride_t, a->T, a->C);
  if (!short_strides({p.res_st, p.block_st, p.gate_st})) return fail(GDP_ERR_UNSUPPORTED, "row strides below 2^31 elements");
  if (partly(p.res, p.res_st, a->residual_out, a->T, a->C, a->residual_dtype)) return fail(GDP_ERR_ALIAS, "residual_out partly overlaps residual");
  const Span residual = rows(p.res, p.res_st, a->C, a->residual_dtype, "residual"), block = rows(p.block, p.block_st, a->C, a->dtype, "block"),
             gate = rows(p.gate, p.gate_st, a->C, a->dtype, "gate"), y = dense(a->y, a->C, a->dtype, "y"),
             out = dense(a->residual_out, a->C, a->residual_dtype, "residual_out");
  if ((st = apart_ok(a->T, {y}, {residual, block, gate, out})) != GDP_OK || (st = apart_ok(a->T, {out}, {block, gate})) != GDP_OK) return st;
  if (a->T == 0) return GDP_OK;
  p.w = a->weight; p.post = a->post_weight; p.scale = a->scale;
  p.y = a->y; p.r = a->residual_out;
  p.T = a->T; p.C = a->C; p.eps = a->eps; p.inv_c = 1.f / (float)a->C;
  p.act = a->activation; p.res_f32 = a->residual_dtype == GDP_DTYPE_F32;
  p.quad_cols = aligned(p.w, 16) && aligned(p.post, 16) && aligned(p.scale, 16);
  const int vec = p.C % kRes == 0 && rows_by(p.res, p.res_st, p.T, a->residual_dtype, 16) && rows_by(p.block, p.block_st, p.T, a->dtype, 16) &&
                  (!p.gate || rows_by(p.gate, p.gate_st, p.T, a->dtype, 16)) && aligned(p.y, 16) && aligned(p.r, 16);
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(a->dtype == GDP_DTYPE_BF16  ? launch_res_fwd<__nv_bfloat16>(p, vec, s)
                     : a->dtype == GDP_DTYPE_F16 ? launch_res_fwd<__half>(p, vec, s)
                                                 : launch_res_fwd<float>(p, vec, s),
                     "residual norm kernel");
}

GDP_EXPORT size_t gdp_residual_norm_workspace_bytes(int64_t T, int64_t C) {
  using namespace gdp::layer;
  if (T < 0 || C < 1 || C > kResMost || T > INT32_MAX) return 0;
  return ((size_t)res_parts(T, C, sm_count()) * 3 * (size_t)C * 4 + 255) / 256 * 256;
}

GDP_EXPORT gdp_status gdp_residual_norm_backward(const gdp_residual_norm_backward_args *a, void *stream) {
  using namespace gdp::layer;
  gdp::set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  gdp_status st = res_ok(a->T, a->C, a->eps, a->dtype, a->residual_dtype, a->activation, a->weight, a->post_weight, a->scale);
  if (st != GDP_OK) return st;
  if ((st = rows_ok(a->d_y, a->d_y_stride_t, a->T, a->C, a->dtype, "d_y")) != GDP_OK) return st;
  if (a->d_residual_out && (st = rows_ok(a->d_residual_out, a->d_residual_out_stride_t, a->T, a->C, a->residual_dtype, "d_residual_out")) != GDP_OK)
    return st;
  if ((st = rows_ok(a->residual_out, a->residual_out_stride_t, a->T, a->C, a->residual_dtype, "residual_out")) != GDP_OK) return st;
  if ((st = rows_ok(a->block, a->block_stride_t, a->T, a->C, a->dtype, "block")) != GDP_OK) return st;
  if (a->gate && (st = rows_ok(a->gate, a->gate_stride_t, a->T, a->C, a->dtype, "gate")) != GDP_OK) return st;
  if ((st = rows_ok(a->d_residual, a->C, a->T, a->C, a->residual_dtype, "d_residual")) != GDP_OK) return st;
  if ((st = rows_ok(a->d_block, a->C, a->T, a->C, a->dtype, "d_block")) != GDP_OK) return st;
  if (a->gate && (st = rows_ok(a->d_gate, a->C, a->T, a->C, a->dtype, "d_gate")) != GDP_OK) return st;
  if (!a->d_weight || (a->post_weight != nullptr) != (a->d_post_weight != nullptr) || (a->scale != nullptr) != (a->d_scale != nullptr))
    return fail(GDP_ERR_INVALID_ARG, "d_weight is required, d_post_weight goes with post_weight and d_scale with scale");
  if (!aligned(a->d_weight, 4) || !aligned(a->d_post_weight, 4) || !aligned(a->d_scale, 4))
    return fail(GDP_ERR_INVALID_ARG, "fp32 buffers must be 4-byte aligned");
  if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < gdp_residual_norm_workspace_bytes(a->T, a->C))
    return fail(GDP_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than gdp_residual_norm_workspace_bytes");
  ResProblem p{};
  p.res = a->residual_out; p.block = a->block; p.gate = a->gate; p.dy = a->d_y; p.dr = a->d_residual_out;
  p.res_st = stride_of(a->residual_out_stride_t, a->T, a->C); p.block_st = stride_of(a->block_stride_t, a->T, a->C);
  p.gate_st = stride_of(a->gate_stride_t, a->T, a->C); p.dy_st = stride_of(a->d_y_stride_t, a->T, a->C);
  p.dr_st = stride_of(a->d_residual_out_stride_t, a->T, a->C);
  if (!short_strides({p.res_st, p.block_st, p.gate_st, p.dy_st, p.dr_st})) return fail(GDP_ERR_UNSUPPORTED, "row strides below 2^31 elements");
  if (partly(p.dr, p.dr_st, a->d_residual, a->T, a->C, a->residual_dtype)) return fail(GDP_ERR_ALIAS, "d_residual partly overlaps d_residual_out");
  const Span dy = rows(p.dy, p.dy_st, a->C, a->dtype, "d_y"), dr = rows(p.dr, p.dr_st, a->C, a->residual_dtype, "d_residual_out"),
             res = rows(p.res, p.res_st, a->C, a->residual_dtype, "residual_out"), block = rows(p.block, p.block_st, a->C, a->dtype, "block"),
             gate = rows(p.gate, p.gate_st, a->C, a->dtype, "gate"), dres = dense(a->d_residual, a->C, a->residual_dtype, "d_residual");
  if ((st = apart_ok(a->T, {dense(a->d_block, a->C, a->dtype, "d_block"), dense(a->gate ? a->d_gate : nullptr, a->C, a->dtype, "d_gate")},
                     {dy, dr, res, block, gate, dres})) != GDP_OK ||
      (st = apart_ok(a->T, {dres}, {dy, res, block, gate})) != GDP_OK)
    return st;
  p.w = a->weight; p.post = a->post_weight; p.scale = a->scale;
  p.dres = a->d_residual; p.dblock = a->d_block; p.dgate = a->d_gate;
  p.partial = static_cast<float *>(a->workspace);
  p.T = a->T; p.C = a->C; p.eps = a->eps; p.inv_c = 1.f / (float)a->C;
  p.act = a->activation; p.res_f32 = a->residual_dtype == GDP_DTYPE_F32;
  p.quad_cols = aligned(p.w, 16) && aligned(p.post, 16) && aligned(p.scale, 16);
  const int vec = p.C % kRes == 0 && rows_by(p.res, p.res_st, p.T, a->residual_dtype, 16) && rows_by(p.block, p.block_st, p.T, a->dtype, 16) &&
                  rows_by(p.dy, p.dy_st, p.T, a->dtype, 16) && (!p.gate || (rows_by(p.gate, p.gate_st, p.T, a->dtype, 16) && aligned(p.dgate, 16))) &&
                  (!p.dr || rows_by(p.dr, p.dr_st, p.T, a->residual_dtype, 16)) && aligned(p.dres, 16) && aligned(p.dblock, 16);
  const int64_t parts = res_parts(p.T, p.C, sm_count());
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = a->dtype == GDP_DTYPE_BF16  ? launch_res_bwd<__nv_bfloat16>(p, vec, parts, s)
                  : a->dtype == GDP_DTYPE_F16 ? launch_res_bwd<__half>(p, vec, parts, s)
                                              : launch_res_bwd<float>(p, vec, parts, s);
  if (e == cudaSuccess) {
    ColumnSums c{};
    c.from = p.partial; c.parts = parts; c.cols = 3 * p.C;
    c.to[0] = a->d_weight; c.to[1] = a->d_post_weight; c.to[2] = a->d_scale;
    c.first[1] = p.C; c.first[2] = 2 * p.C; c.first[3] = c.cols;
    e = launch_column_sums(c, s);
  }
  return cuda_status(e, "residual norm backward kernels");
}

GDP_EXPORT size_t gdp_block_args_size(int which) {
  switch (which) {
    case 0: return sizeof(gdp_conv_args);
    case 1: return sizeof(gdp_conv_backward_args);
    case 2: return sizeof(gdp_scan_args);
    case 3: return sizeof(gdp_scan_backward_args);
    case 4: return sizeof(gdp_residual_norm_args);
    case 5: return sizeof(gdp_residual_norm_backward_args);
    default: return 0;
  }
}
