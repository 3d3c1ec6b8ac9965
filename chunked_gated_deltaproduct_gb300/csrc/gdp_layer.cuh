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

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 x, y, z, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 w, x, y, z;\nmov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 x, y, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmul.rn.f32x2 w, x, y;\nmov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 x, y, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 w, x, y;\nmov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// sigmoid(x) and 1 - sigmoid(x) = e^-x sigmoid(x), each to its own relative precision.  e^-x is held to the
// largest fp32 value, so that the second is finite; the first reaches 0 (at x below -87.3, 2^-126), so that its
// product with any finite x does too.  Where it is 0 the second is 0 as well, and not 1: a caller multiplies it by
// the first, or by x and then by the first.
__device__ __forceinline__ void sigmoid_halves(float2 x, float2 *q, float2 *rest) {
  const float2 t = mul2(x, both(-kLog2e));
  float2 e = make_float2(ex2(t.x), ex2(t.y));
  asm("min.NaN.f32 %0, %0, 0f7F7FFFFF;" : "+f"(e.x));
  asm("min.NaN.f32 %0, %0, 0f7F7FFFFF;" : "+f"(e.y));
  const float2 d = add2(e, both(1.f));
  *q = make_float2(rcp(d.x), rcp(d.y));
  *rest = mul2(e, *q);
}

// Two stored values in one register (16-bit types), widened, and back.
template <typename T>
__device__ __forceinline__ float2 widen(uint32_t v);
template <>
__device__ __forceinline__ float2 widen<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 widen<__half>(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
template <typename T>
__device__ __forceinline__ uint32_t narrow(float2 v);
template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(float2 v) {
  const __nv_bfloat162 h = __float22bfloat162_rn(v);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow<__half>(float2 v) {
  const __half2 h = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t *>(&h);
}

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

// Largest absolute value as its bits: they order like the values, with infinities and NaN on top.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Inverse scale of a checkpoint block from its largest absolute value: 127 / amax cut to four
// significant bits (its product with a 16-bit value is exact in fp32, so the codes do not depend on
// the arithmetic), 0 for a block of zeros or next to it.  T: the type the value came from.  Of the
// 16-bit types' values, 127 / amax is a four-bit number only where amax is 127 times a power of two,
// and otherwise at least 2^-15 relative away from one (amax times the number is an integer of at most
// 15 bits); so the approximate reciprocal (2^-22), raised by 2^-20, is cut to the same four bits.
template <typename T>
__device__ __forceinline__ float block_inverse(uint32_t amax_bits) {
  const float amax = __uint_as_float(amax_bits);
  // (amax / 256, so that the largest values' reciprocals are not flushed to zero)
  const float quotient = sizeof(T) == 4 ? __fdiv_rn(127.f, amax) : rcp(amax * 0x1p-8f) * (127.f * 0x1p-8f * (1.f + 0x1p-20f));
  const bool plain = amax >= kTinyAmax && amax_bits < 0x7f800000u;
  return plain ? __uint_as_float(__float_as_uint(quotient) & 0xfff00000u) : 0.f;
}
// 1 / inverse, correctly rounded: the inverse is (8 + i) / 8 times a power of two.
__constant__ const float kEighths[8] = {8.f / 8.f, 8.f / 9.f, 8.f / 10.f, 8.f / 11.f, 8.f / 12.f, 8.f / 13.f, 8.f / 14.f, 8.f / 15.f};
__device__ __forceinline__ float block_scale(uint32_t amax_bits, float inverse) {
  const uint32_t b = __float_as_uint(inverse);
  // 127 / amax is at least 1.875 2^-122; a code of 120 times that one's reciprocal would be 2^128, beyond fp32, for
  // a block whose largest value is the type's: the next number below it makes that the largest fp32 value
  const float s = fminf(kEighths[b >> 20 & 7u] * __uint_as_float((254u << 23) - (b & 0x7f800000u)), __uint_as_float(0x7c088888u));
  return amax_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : b == 0u ? 0.f : s;
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
