// gdp_group_norm.cu -- the grouped norm's C entries, argument checks and column-sum kernel
// (gdp_layer.h; the kernels over rows are in gdp_norm_body.cuh).
#include "gdp_norm.cuh"

namespace gdp {
namespace layer {
namespace {

// Adds up the parts of every column in a fixed order: 32 columns per CTA, each warp a stride of the
// parts, then the warps' sums in turn.
constexpr int kFinishWarps = 32;
__global__ void __launch_bounds__(32 * kFinishWarps) gdp_norm_finish_kernel(const float *partial, int64_t parts, int64_t cols, float *dw,
                                                                            float *db) {
  __shared__ float sums[kFinishWarps][32];
  sm100::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const float *from = partial + (blockIdx.y ? parts * cols : 0);
  float s = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int64_t i = warp; i < parts; i += kFinishWarps) s += from[i * cols + col];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kFinishWarps; ++i) s += sums[i][lane];
    (blockIdx.y ? db : dw)[col] = s;
  }
}

// Eight channels at a time: whole chunks of 16 bytes in every tensor.
bool vec_ok(const void *p, int64_t st, int64_t sh, int64_t T, int64_t H, int type) {
  return aligned(p, 16) && (T <= 1 || st * dtype_size(type) % 16 == 0) && (H <= 1 || sh * dtype_size(type) % 16 == 0);
}

gdp_status norm_status(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return GDP_OK;
  set_last_error("%s: %s", what, cudaGetErrorString(e));
  return GDP_ERR_CUDA;
}

gdp_status check_norm(int64_t T, int64_t H, int64_t D, float eps, int type, int act, bool has_gate, const float *w) {
  if (T < 0 || H < 1 || D < 1) return fail(GDP_ERR_INVALID_ARG, "T >= 0, H >= 1 and D >= 1 are required");
  if (D > 8192 || H > (1 << 20) || T > INT32_MAX) return fail(GDP_ERR_UNSUPPORTED, "D up to 8192, H up to 2^20, T below 2^31");
  if (!dtype_ok(type)) return fail(GDP_ERR_UNSUPPORTED, "dtype must be GDP_DTYPE_BF16, GDP_DTYPE_F16 or GDP_DTYPE_F32");
  if (!(eps >= 0.f)) return fail(GDP_ERR_INVALID_ARG, "eps must not be negative");
  if (act != GDP_ACT_NONE && act != GDP_ACT_SILU && act != GDP_ACT_SIGMOID)
    return fail(GDP_ERR_INVALID_ARG, "activation must be GDP_ACT_NONE, GDP_ACT_SILU or GDP_ACT_SIGMOID");
  // (of an empty batch the gate may be given and have no address)
  if (T > 0 && has_gate && act == GDP_ACT_NONE) return fail(GDP_ERR_INVALID_ARG, "z needs an activation");
  if (T > 0 && !has_gate && act == GDP_ACT_SIGMOID) return fail(GDP_ERR_INVALID_ARG, "the sigmoid activation gates with z");
  if (!w) return fail(GDP_ERR_INVALID_ARG, "weight is required");
  return GDP_OK;
}

gdp_status check_heads(const void *p, int64_t st, int64_t sh, int64_t T, int64_t H, int64_t D, int type, const char *name) {
  if (T > 0 && !p) {
    set_last_error("%s is required", name);
    return GDP_ERR_INVALID_ARG;
  }
  if (!aligned(p, dtype_size(type)) || (T > 1 && st < 1) || (H > 1 && sh < D)) {
    set_last_error("%s must be aligned to its elements, with a positive token stride and heads at least D apart", name);
    return GDP_ERR_INVALID_ARG;
  }
  return GDP_OK;
}

}  // namespace
}  // namespace layer
}  // namespace gdp

GDP_EXPORT gdp_status gdp_group_norm(const gdp_group_norm_args *a, void *stream) {
  using namespace gdp::layer;
  gdp::set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  gdp_status st = check_norm(a->T, a->H, a->D, a->eps, a->dtype, a->activation, a->z != nullptr, a->weight);
  if (st != GDP_OK) return st;
  if ((st = check_heads(a->o, a->o_stride_t, a->o_stride_h, a->T, a->H, a->D, a->dtype, "o")) != GDP_OK) return st;
  if (a->z && (st = check_heads(a->z, a->z_stride_t, a->z_stride_h, a->T, a->H, a->D, a->dtype, "z")) != GDP_OK) return st;
  if ((st = check_heads(a->y, a->H * a->D, a->D, a->T, a->H, a->D, a->dtype, "y")) != GDP_OK) return st;
  if ((a->o_codes != nullptr) != (a->o_scales != nullptr) || (a->z_codes != nullptr) != (a->z_scales != nullptr) ||
      (a->z_codes && !a->z))
    return fail(GDP_ERR_INVALID_ARG, "a checkpoint needs its codes and its scales, z's also z");
  if (!aligned(a->o_scales, 4) || !aligned(a->z_scales, 4) || !aligned(a->weight, 4) || !aligned(a->bias, 4))
    return fail(GDP_ERR_INVALID_ARG, "fp32 buffers must be 4-byte aligned");
  if (a->T == 0) return GDP_OK;
  NormProblem p{};
  p.o = a->o; p.o_st = a->o_stride_t; p.o_sh = a->o_stride_h;
  p.z = a->z; p.z_st = a->z_stride_t; p.z_sh = a->z_stride_h;
  p.w = a->weight; p.b = a->bias; p.y = a->y;
  p.o_codes = a->o_codes; p.o_scales = a->o_scales; p.z_codes = a->z_codes; p.z_scales = a->z_scales;
  p.T = a->T; p.H = a->H; p.D = a->D; p.eps = a->eps;
  p.inv_d = 1.f / (float)p.D;
  p.center = a->center != 0; p.per_head = a->per_head != 0; p.act = a->activation;
  const int vec = p.D % 8 == 0 && vec_ok(p.o, p.o_st, p.o_sh, p.T, p.H, a->dtype) && (!p.z || vec_ok(p.z, p.z_st, p.z_sh, p.T, p.H, a->dtype)) &&
                  aligned(p.y, 16) && aligned(p.o_codes, 8) && aligned(p.z_codes, 8);
  const NormPlan n = norm_plan(p.T, p.H, p.D, p.per_head, vec, sm_count(), kNormFwdCtas);
  p.vec_cols = p.D % 8 == 0 && aligned(p.w, 16) && aligned(p.b, 16);
  p.heads = n.heads; p.groups = n.groups; p.parts = n.parts;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = a->dtype == GDP_DTYPE_BF16  ? launch_norm_fwd<__nv_bfloat16>(p, n, s)
                        : a->dtype == GDP_DTYPE_F16 ? launch_norm_fwd<__half>(p, n, s)
                                                    : launch_norm_fwd<float>(p, n, s);
  return norm_status(e, "group norm kernel");
}

GDP_EXPORT size_t gdp_group_norm_workspace_bytes(int64_t T, int64_t H, int64_t D, int per_head) {
  using namespace gdp::layer;
  if (T < 0 || H < 1 || D < 1 || D > 8192 || H > (1 << 20) || T > INT32_MAX) return 0;
  const size_t cols = per_head ? (size_t)(H * D) : (size_t)D;
  const int64_t a = norm_plan(T, H, D, per_head, 0, sm_count(), kNormBwdCtas).parts, b = norm_plan(T, H, D, per_head, 1, sm_count(), kNormBwdCtas).parts;
  return ((size_t)(a > b ? a : b) * 2 * cols * 4 + 255) / 256 * 256;
}

GDP_EXPORT gdp_status gdp_group_norm_backward(const gdp_group_norm_backward_args *a, void *stream) {
  using namespace gdp::layer;
  gdp::set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  const bool zed = a->z || a->z_codes;
  gdp_status st = check_norm(a->T, a->H, a->D, a->eps, a->dtype, a->activation, zed, a->weight);
  if (st != GDP_OK) return st;
  if (a->T > 0 && (a->o != nullptr) == (a->o_codes != nullptr))
    return fail(GDP_ERR_INVALID_ARG, "exactly one of o and o_codes is required");
  if (a->z && a->z_codes) return fail(GDP_ERR_INVALID_ARG, "z is given either as a tensor or as codes");
  if (zed && (a->z != nullptr) != (a->o != nullptr)) return fail(GDP_ERR_INVALID_ARG, "o and z are both tensors or both codes");
  if ((st = check_heads(a->d_y, a->d_y_stride_t, a->d_y_stride_h, a->T, a->H, a->D, a->dtype, "d_y")) != GDP_OK) return st;
  if (a->o && (st = check_heads(a->o, a->o_stride_t, a->o_stride_h, a->T, a->H, a->D, a->dtype, "o")) != GDP_OK) return st;
  if (a->z && (st = check_heads(a->z, a->z_stride_t, a->z_stride_h, a->T, a->H, a->D, a->dtype, "z")) != GDP_OK) return st;
  if ((a->o_codes && !a->o_scales) || (a->z_codes && !a->z_scales))
    return fail(GDP_ERR_INVALID_ARG, "codes need their scales");
  if ((st = check_heads(a->d_o, a->H * a->D, a->D, a->T, a->H, a->D, a->dtype, "d_o")) != GDP_OK) return st;
  if (zed && (st = check_heads(a->d_z, a->H * a->D, a->D, a->T, a->H, a->D, a->dtype, "d_z")) != GDP_OK) return st;
  if (!a->d_weight || (a->bias != nullptr) != (a->d_bias != nullptr))
    return fail(GDP_ERR_INVALID_ARG, "d_weight is required, d_bias goes with bias");
  if (!aligned(a->o_scales, 4) || !aligned(a->z_scales, 4) || !aligned(a->weight, 4) || !aligned(a->bias, 4) ||
      !aligned(a->d_weight, 4) || !aligned(a->d_bias, 4))
    return fail(GDP_ERR_INVALID_ARG, "fp32 buffers must be 4-byte aligned");
  if (!a->workspace || !aligned(a->workspace, 256) ||
      a->workspace_bytes < gdp_group_norm_workspace_bytes(a->T, a->H, a->D, a->per_head))
    return fail(GDP_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than gdp_group_norm_workspace_bytes");
  NormProblem p{};
  p.o = a->o; p.o_st = a->o_stride_t; p.o_sh = a->o_stride_h;
  p.z = a->z; p.z_st = a->z_stride_t; p.z_sh = a->z_stride_h;
  p.o_codes_in = a->o_codes; p.o_scales_in = a->o_scales; p.z_codes_in = a->z_codes; p.z_scales_in = a->z_scales;
  p.w = a->weight; p.b = a->bias;
  p.dy = a->d_y; p.dy_st = a->d_y_stride_t; p.dy_sh = a->d_y_stride_h;
  p.d_o = a->d_o; p.d_z = a->d_z; p.dw = a->d_weight; p.db = a->d_bias;
  p.T = a->T; p.H = a->H; p.D = a->D; p.eps = a->eps;
  p.inv_d = 1.f / (float)p.D;
  p.center = a->center != 0; p.per_head = a->per_head != 0; p.act = a->activation;
  p.partial = static_cast<float *>(a->workspace);
  cudaStream_t s = (cudaStream_t)stream;
  const int vec = p.D % 8 == 0 && vec_ok(p.dy, p.dy_st, p.dy_sh, p.T, p.H, a->dtype) &&
                  (!p.o || vec_ok(p.o, p.o_st, p.o_sh, p.T, p.H, a->dtype)) && (!p.z || vec_ok(p.z, p.z_st, p.z_sh, p.T, p.H, a->dtype)) &&
                  aligned(p.o_codes_in, 8) && aligned(p.z_codes_in, 8) && aligned(p.d_o, 16) && aligned(p.d_z, 16);
  const NormPlan n = norm_plan(p.T, p.H, p.D, p.per_head, vec, sm_count(), kNormBwdCtas);
  p.vec_cols = p.D % 8 == 0 && aligned(p.w, 16) && aligned(p.b, 16);
  p.heads = n.heads; p.groups = n.groups; p.parts = n.parts;
  cudaError_t e = a->dtype == GDP_DTYPE_BF16  ? launch_norm_bwd<__nv_bfloat16>(p, n, s)
                  : a->dtype == GDP_DTYPE_F16 ? launch_norm_bwd<__half>(p, n, s)
                                              : launch_norm_bwd<float>(p, n, s);
  if (e == cudaSuccess) {
    const int64_t cols = p.per_head ? p.H * p.D : p.D;
    e = gdp::launch_kernel(gdp_norm_finish_kernel, dim3((unsigned)((cols + 31) / 32), p.db ? 2 : 1), dim3(32 * kFinishWarps), 0, s, true,
                           (const float *)p.partial, n.parts, cols, p.dw, p.db);
  }
  return norm_status(e, "group norm backward kernels");
}
