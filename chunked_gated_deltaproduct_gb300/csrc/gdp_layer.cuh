// gdp_layer.cuh -- what the layer operators (gdp_layer.h) share: element types, gates,
// activations, the 8-bit checkpoint blocks and the host's checks.
#pragma once

#include "../../include/gdp_layer.h"
#include "gdp_internal.cuh"

namespace gdp {
namespace layer {

constexpr int kBlock = 128;                  // channels that share one scale of an 8-bit checkpoint
constexpr float kTinyAmax = 0x1p-100f;       // a block below this is stored as zeros (127 / amax stays finite)

// ---- element types: T is float, __nv_bfloat16 or __half ----
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// e^x by the hardware's base-2 exponential: relative error about 2^-22 + |x| 2^-24, 0 below 2^-126.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * kLog2e));
  return y;
}

// Decay a and input factor f of gate value g (b = f x).  The sigmoid's two halves come from the same
// exponential of -|g|, so that 1 - a keeps its relative precision where a is near one.
template <int GATE>
__device__ __forceinline__ void gate_eval(float g, float *a, float *f) {
  if (GATE == GDP_GATE_LOG) {
    *a = exp_fast(g);
    *f = 1.f;
  } else if (GATE == GDP_GATE_ALPHA) {
    *a = g;
    *f = 1.f;
  } else {
    const float e = exp_fast(-fabsf(g)), big = __fdividef(1.f, 1.f + e), small = e * big;
    *a = g >= 0.f ? big : small;
    *f = g >= 0.f ? small : big;
    if (g != g) *a = *f = g;
  }
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + exp_fast(-z)); }

// Largest absolute value as its bits: they order like the values, with infinities and NaN on top.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Inverse scale of a checkpoint block from its largest absolute value: 127 / amax cut to four
// significant bits (its product with a 16-bit value is exact in fp32, so the codes do not depend on
// the arithmetic), 0 for a block of zeros or next to it.
__device__ __forceinline__ float block_inverse(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 0.f;
  const float amax = __uint_as_float(amax_bits);
  if (amax < kTinyAmax) return 0.f;
  return __uint_as_float(__float_as_uint(__fdiv_rn(127.f, amax)) & 0xfff00000u);
}
__device__ __forceinline__ float block_scale(uint32_t amax_bits, float inverse) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return inverse > 0.f ? __fdiv_rn(1.f, inverse) : 0.f;
}
// round-to-even(v k) as a signed byte: v k + 1.5 2^23 in one rounding leaves the integer in the low
// bits.  A zero inverse gives code 0 whatever v is (0 times an infinity would be NaN).
__device__ __forceinline__ uint32_t block_code(float v, float inverse) {
  return inverse > 0.f ? (__float_as_uint(fmaf(v, inverse, 12582912.f)) & 0xffu) : 0u;
}

// ---- host side ----
inline int dtype_size(int t) { return t == GDP_DTYPE_F32 ? 4 : 2; }
inline bool dtype_ok(int t) { return t == GDP_DTYPE_F32 || t == GDP_DTYPE_BF16 || t == GDP_DTYPE_F16; }
inline gdp_status fail(gdp_status st, const char *why) {
  set_last_error("%s", why);
  return st;
}
inline gdp_status launch_status(const char *what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return GDP_OK;
  set_last_error("%s: %s", what, cudaGetErrorString(e));
  return GDP_ERR_CUDA;
}
inline bool aligned(const void *p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
inline bool overlap(const void *a, const void *b, size_t bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + bytes && y < x + bytes;
}
// Neither the same range nor disjoint.
inline bool partly_overlap(const void *a, const void *b, size_t bytes) {
  return a != b && overlap(a, b, bytes);
}

}  // namespace layer
}  // namespace gdp

#define GDP_EXPORT extern "C" __attribute__((visibility("default")))
