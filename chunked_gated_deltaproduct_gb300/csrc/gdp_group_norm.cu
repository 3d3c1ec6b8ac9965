// gdp_group_norm.cu -- the grouped norm with an activated gate, its 8-bit checkpoints and its
// backward pass (gdp_layer.h).
//
// One warp per (token, head) row of D channels.  The sums over rows of the backward pass (dweight,
// dbias) run in a fixed order: column sums of a slab of rows into the workspace, then the slabs in turn.
#include "gdp_layer.cuh"

namespace gdp {
namespace layer {
namespace {

constexpr int kWarps = 8;
constexpr int kSlabs = 256;  // row slabs of the column sums

struct NormProblem {
  const void *o, *z;
  int64_t o_st, o_sh, z_st, z_sh;
  const int8_t *o_codes_in, *z_codes_in;  // backward: read instead of o and z
  const float *o_scales_in, *z_scales_in;
  const float *w, *b;
  void *y;
  int8_t *o_codes, *z_codes;
  float *o_scales, *z_scales;
  const void *dy;
  int64_t dy_st, dy_sh;
  void *d_o, *d_z;
  float *dw, *db, *stats, *partial;
  int64_t T, H, D;
  float eps;
  int type, center, per_head, act;
};

__device__ __forceinline__ float load_any(const void *p, int64_t i, int type) {
  if (type == GDP_DTYPE_F32) return static_cast<const float *>(p)[i];
  if (type == GDP_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  return __half2float(static_cast<const __half *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int64_t i, int type, float v) {
  if (type == GDP_DTYPE_F32) static_cast<float *>(p)[i] = v;
  else if (type == GDP_DTYPE_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half *>(p)[i] = __float2half_rn(v);
}
__device__ __forceinline__ float warp_sum(float v) {
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// Element d of row (t, h) of o or z, from the tensor or its checkpoint.
struct RowReader {
  const void *p;
  const int8_t *codes;
  const float *scales;
  int64_t at, row, D;
  int type;
  __device__ float operator()(int64_t d) const {
    if (codes) return codes[row * D + d] * scales[row * ((D + kBlock - 1) / kBlock) + d / kBlock];
    return load_any(p, at + d, type);
  }
};
__device__ __forceinline__ RowReader reader_o(const NormProblem &p, int64_t t, int64_t h) {
  return {p.o, p.o_codes_in, p.o_scales_in, t * p.o_st + h * p.o_sh, t * p.H + h, p.D, p.type};
}
__device__ __forceinline__ RowReader reader_z(const NormProblem &p, int64_t t, int64_t h) {
  return {p.z, p.z_codes_in, p.z_scales_in, t * p.z_st + h * p.z_sh, t * p.H + h, p.D, p.type};
}
__device__ __forceinline__ bool has_z(const NormProblem &p) { return p.z || p.z_codes_in; }

__device__ __forceinline__ void row_stats(const NormProblem &p, const RowReader &o, int lane, float *mean, float *rstd) {
  float s = 0.f, m = 0.f;
  if (p.center) {
    for (int64_t d = lane; d < p.D; d += 32) s += o(d);
    m = warp_sum(s) / (float)p.D;
  }
  s = 0.f;
  for (int64_t d = lane; d < p.D; d += 32) s += (o(d) - m) * (o(d) - m);
  *mean = m;
  *rstd = rsqrtf(warp_sum(s) / (float)p.D + p.eps);
}

// act(t) and its slope at t.
__device__ __forceinline__ void activation(int act, float t, float *v, float *slope) {
  float q, r;  // sigmoid(t) and 1 - sigmoid(t), each to its own relative precision
  gate_eval<GDP_GATE_SIGMOID>(t, &q, &r);
  *v = act == GDP_ACT_SILU ? t * q : q;
  *slope = act == GDP_ACT_SILU ? q * (1.f + t * r) : q * r;
}

__device__ __forceinline__ void save_row(const RowReader &v, int64_t row, int64_t D, int8_t *codes, float *scales, int lane) {
  const int64_t nb = (D + kBlock - 1) / kBlock;
  for (int64_t b = 0; b < nb; ++b) {
    const int64_t lo = b * kBlock, hi = min(lo + kBlock, D);
    uint32_t amax = 0;
    for (int64_t d = lo + lane; d < hi; d += 32) amax = max(amax, abs_bits(v(d)));
    amax = __reduce_max_sync(0xffffffffu, amax);
    const float inv = block_inverse(amax);
    for (int64_t d = lo + lane; d < hi; d += 32) codes[row * D + d] = (int8_t)block_code(v(d), inv);
    if (lane == 0) scales[row * nb + b] = block_scale(amax, inv);
  }
}

__global__ void __launch_bounds__(kWarps * 32) gdp_norm_fwd_kernel(NormProblem p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.T * p.H) return;
  const int64_t t = row / p.H, h = row % p.H;
  const RowReader o = reader_o(p, t, h), z = reader_z(p, t, h);
  float mean, rstd;
  row_stats(p, o, lane, &mean, &rstd);
  const float *w = p.w + (p.per_head ? h * p.D : 0), *b = p.b ? p.b + (p.per_head ? h * p.D : 0) : nullptr;
  for (int64_t d = lane; d < p.D; d += 32) {
    const float u = (o(d) - mean) * rstd * w[d] + (b ? b[d] : 0.f);
    float v = 1.f, slope;
    if (has_z(p)) {
      activation(p.act, z(d), &v, &slope);
      if (p.act == GDP_ACT_NONE) v = 1.f;
    } else if (p.act == GDP_ACT_SILU) {
      v = sigmoid(u);
    }
    store_any(p.y, row * p.D + d, p.type, u * v);
  }
  if (p.o_codes) save_row(o, row, p.D, p.o_codes, p.o_scales, lane);
  if (p.z_codes) save_row(z, row, p.D, p.z_codes, p.z_scales, lane);
}

// du and dz of one element from u, z and dy.
__device__ __forceinline__ void through_gate(const NormProblem &p, float u, float z, float dy, float *du, float *dz) {
  float v, slope;
  *du = dy;
  *dz = 0.f;
  if (p.act == GDP_ACT_NONE) return;
  activation(p.act, has_z(p) ? z : u, &v, &slope);
  if (has_z(p)) {
    *du = dy * v;
    *dz = dy * u * slope;
  } else {
    *du = dy * slope;
  }
}

__global__ void __launch_bounds__(kWarps * 32) gdp_norm_bwd_kernel(NormProblem p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.T * p.H) return;
  const int64_t t = row / p.H, h = row % p.H;
  const RowReader o = reader_o(p, t, h), z = reader_z(p, t, h);
  const bool zed = has_z(p);
  float mean, rstd;
  row_stats(p, o, lane, &mean, &rstd);
  if (lane == 0) {
    p.stats[2 * row] = mean;
    p.stats[2 * row + 1] = rstd;
  }
  const float *w = p.w + (p.per_head ? h * p.D : 0), *b = p.b ? p.b + (p.per_head ? h * p.D : 0) : nullptr;
  const int64_t at = t * p.dy_st + h * p.dy_sh;
  float s1 = 0.f, s2 = 0.f;
  for (int64_t d = lane; d < p.D; d += 32) {
    const float n = (o(d) - mean) * rstd;
    float du, dz;
    through_gate(p, n * w[d] + (b ? b[d] : 0.f), zed ? z(d) : 0.f, load_any(p.dy, at + d, p.type), &du, &dz);
    if (zed) store_any(p.d_z, row * p.D + d, p.type, dz);
    s1 += du * w[d];
    s2 += du * w[d] * n;
  }
  s1 = p.center ? warp_sum(s1) / (float)p.D : 0.f;
  s2 = warp_sum(s2) / (float)p.D;
  for (int64_t d = lane; d < p.D; d += 32) {
    const float n = (o(d) - mean) * rstd;
    float du, dz;
    through_gate(p, n * w[d] + (b ? b[d] : 0.f), zed ? z(d) : 0.f, load_any(p.dy, at + d, p.type), &du, &dz);
    store_any(p.d_o, row * p.D + d, p.type, rstd * (du * w[d] - s1 - n * s2));
  }
}

// Column sums of slab blockIdx.y: partial[slab][0] = sum du n, [1] = sum du.
__global__ void __launch_bounds__(128) gdp_norm_columns_kernel(NormProblem p) {
  const int64_t cols = p.per_head ? p.H * p.D : p.D, col = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (col >= cols) return;
  const int64_t h0 = p.per_head ? col / p.D : 0, d = col % p.D, step = p.per_head ? p.H : 1;
  const int64_t rows = p.per_head ? p.T : p.T * p.H, lo = rows * blockIdx.y / kSlabs, hi = rows * (blockIdx.y + 1) / kSlabs;
  float sw = 0.f, sb = 0.f;
  for (int64_t r = lo; r < hi; ++r) {
    const int64_t row = r * step + h0, t = row / p.H, h = row % p.H;
    const float n = (reader_o(p, t, h)(d) - p.stats[2 * row]) * p.stats[2 * row + 1];
    float du, dz;
    through_gate(p, n * p.w[col] + (p.b ? p.b[col] : 0.f), has_z(p) ? reader_z(p, t, h)(d) : 0.f,
                 load_any(p.dy, t * p.dy_st + h * p.dy_sh + d, p.type), &du, &dz);
    sw += du * n;
    sb += du;
  }
  p.partial[(2 * blockIdx.y) * cols + col] = sw;
  p.partial[(2 * blockIdx.y + 1) * cols + col] = sb;
}

__global__ void __launch_bounds__(128) gdp_norm_finish_kernel(NormProblem p) {
  const int64_t cols = p.per_head ? p.H * p.D : p.D, col = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (col >= cols) return;
  float sw = 0.f, sb = 0.f;
  for (int s = 0; s < kSlabs; ++s) {
    sw += p.partial[(2 * s) * cols + col];
    sb += p.partial[(2 * s + 1) * cols + col];
  }
  p.dw[col] = sw;
  if (p.db) p.db[col] = sb;
}

gdp_status check_norm(int64_t T, int64_t H, int64_t D, float eps, int type, int act, bool has_gate, const float *w) {
  if (T < 0 || H < 1 || D < 1) return fail(GDP_ERR_INVALID_ARG, "T >= 0, H >= 1 and D >= 1 are required");
  if (D > 8192 || H > (1 << 20) || T > INT32_MAX) return fail(GDP_ERR_UNSUPPORTED, "D up to 8192, H up to 2^20, T below 2^31");
  if (!dtype_ok(type)) return fail(GDP_ERR_UNSUPPORTED, "dtype must be GDP_DTYPE_BF16, GDP_DTYPE_F16 or GDP_DTYPE_F32");
  if (!(eps >= 0.f)) return fail(GDP_ERR_INVALID_ARG, "eps must not be negative");
  if (act != GDP_ACT_NONE && act != GDP_ACT_SILU && act != GDP_ACT_SIGMOID)
    return fail(GDP_ERR_INVALID_ARG, "activation must be GDP_ACT_NONE, GDP_ACT_SILU or GDP_ACT_SIGMOID");
  if (has_gate && act == GDP_ACT_NONE) return fail(GDP_ERR_INVALID_ARG, "z needs an activation");
  if (!has_gate && act == GDP_ACT_SIGMOID) return fail(GDP_ERR_INVALID_ARG, "the sigmoid activation gates with z");
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
  p.type = a->dtype; p.center = a->center != 0; p.per_head = a->per_head != 0; p.act = a->activation;
  const int64_t blocks = (p.T * p.H + kWarps - 1) / kWarps;
  if (blocks > INT32_MAX) return fail(GDP_ERR_UNSUPPORTED, "too many rows for one launch");
  gdp_norm_fwd_kernel<<<(unsigned)blocks, kWarps * 32, 0, (cudaStream_t)stream>>>(p);
  return launch_status("group norm kernel");
}

GDP_EXPORT size_t gdp_group_norm_workspace_bytes(int64_t T, int64_t H, int64_t D, int per_head) {
  using namespace gdp::layer;
  if (T < 0 || H < 1 || D < 1 || D > 8192 || H > (1 << 20) || T > INT32_MAX) return 0;
  const size_t cols = per_head ? (size_t)(H * D) : (size_t)D;
  return ((size_t)(T * H) * 8 + 255) / 256 * 256 + (size_t)kSlabs * 2 * cols * 4 + 256;
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
  p.type = a->dtype; p.center = a->center != 0; p.per_head = a->per_head != 0; p.act = a->activation;
  p.stats = static_cast<float *>(a->workspace);
  p.partial = p.stats + ((size_t)(p.T * p.H) * 2 + 63) / 64 * 64;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t blocks = (p.T * p.H + kWarps - 1) / kWarps, cols = p.per_head ? p.H * p.D : p.D;
  if (blocks > INT32_MAX) return fail(GDP_ERR_UNSUPPORTED, "too many rows for one launch");
  if (blocks > 0) gdp_norm_bwd_kernel<<<(unsigned)blocks, kWarps * 32, 0, s>>>(p);
  const dim3 grid((unsigned)((cols + 127) / 128), kSlabs);
  gdp_norm_columns_kernel<<<grid, 128, 0, s>>>(p);
  gdp_norm_finish_kernel<<<grid.x, 128, 0, s>>>(p);
  return launch_status("group norm backward kernels");
}
