// gdp_norm_body.cuh -- the grouped norm with an activated gate: forward (with 8-bit checkpoints) and
// backward kernels (gdp_layer.h).
//
// A row (token, head) is held by a group of threads, eight channels per thread and chunk: 8, 16 or 32
// lanes of a warp (D up to 64, 128, 256), or a whole CTA.  A group keeps one head, so that its weights
// stay in registers and the backward's sums over tokens (dweight, dbias) accumulate there; it walks
// over tokens with the next row's loads in flight.  Those sums leave once per CTA (or per group where
// every head has its own weights) and a second kernel adds them up in a fixed order.
#pragma once

#include "gdp_norm.cuh"

#ifndef FWDB
#define FWDB 4
#define BWDB 3
#endif
namespace gdp {
namespace layer {
namespace {

// Eight values of a row as they lie in memory.
template <typename T>
struct alignas(8 * sizeof(T) > 16 ? 16 : 8 * sizeof(T)) Eight {
  T v[8];
  __device__ __forceinline__ uint32_t word(int i) const { return reinterpret_cast<const uint32_t *>(v)[i]; }
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (sizeof(T) == 4) return make_float2(v[2 * i], v[2 * i + 1]);
    else return widen<T>(word(i));
  }
  __device__ __forceinline__ void set(int i, float2 x) {
    if constexpr (sizeof(T) == 4) {
      v[2 * i] = x.x;
      v[2 * i + 1] = x.y;
    } else {
      reinterpret_cast<uint32_t *>(v)[i] = narrow<T>(x);
    }
  }
};
// Source of o and z: a tensor, or codes with the scales of the (one or two) blocks the eight lie in.
template <typename T, bool Q8, bool VEC>
struct Source {
  Eight<typename std::conditional<Q8, int8_t, T>::type> e;
  float scale[Q8 ? (VEC ? 1 : 2) : 1];
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (Q8) {
      // a byte plus 128 under the exponent of 2^23 is 2^23 + 128 + code
      const uint32_t w = e.word(i >> 1) ^ 0x80808080u;
      const float2 m = make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + (i & 1) * 2)),
                                   __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441 + (i & 1) * 2)));
      return mul2(add2(m, both(-8388736.f)), both(scale[VEC ? 0 : i >> 1]));
    } else {
      return e.pair(i);
    }
  }
};

// Where a thread's channels lie in its row.  VEC: eight consecutive ones; else eight 32 apart, so that a
// warp's accesses stay one run of memory.  Either way a checkpoint block of 128 channels lies in one warp:
// in 16 lanes (VEC), or in four of the eight of all 32.
template <bool VEC, int L>
struct Place {
  int id, first, width;  // thread of the group, first channel of chunk 0, channels of a chunk of the whole group
  __device__ __forceinline__ Place() {
    id = L > 0 ? (int)threadIdx.x % (L > 0 ? L : 1) : (int)threadIdx.x;
    width = (L > 0 ? L : (int)blockDim.x) * 8;
    first = VEC ? id * 8 : (id >> 5) * 256 + (id & 31);
  }
  __device__ __forceinline__ int at(int k, int j) const { return k * width + first + (VEC ? j : 32 * j); }
};

template <typename T, bool VEC, int L>
__device__ __forceinline__ void load_eight(Eight<T> &e, const T *row, const Place<VEC, L> &pl, int k, int D, bool on) {
  if constexpr (VEC) {
    using V = typename std::conditional<sizeof(T) == 1, uint2, uint4>::type;
    constexpr int n = (int)(8 * sizeof(T) / sizeof(V));
    V *to = reinterpret_cast<V *>(e.v);
    const bool in = on && pl.at(k, 0) < D;
#pragma unroll
    for (int i = 0; i < n; ++i) to[i] = in ? __ldcs(reinterpret_cast<const V *>(row + pl.at(k, 0)) + i) : V{};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = on && pl.at(k, j) < D;
      if constexpr (sizeof(T) == 1) e.v[j] = in ? row[pl.at(k, j)] : (T)0;
      else e.v[j] = in ? row[pl.at(k, j)] : from_f32<T>(0.f);
    }
  }
}
template <typename T, bool VEC, int L>
__device__ __forceinline__ void store_eight(T *row, const Eight<T> &e, const Place<VEC, L> &pl, int k, int D) {
  if constexpr (VEC) {
    using V = typename std::conditional<sizeof(T) == 1, uint2, uint4>::type;
    constexpr int n = (int)(8 * sizeof(T) / sizeof(V));
    if (pl.at(k, 0) < D) {
#pragma unroll
      for (int i = 0; i < n; ++i) __stcs(reinterpret_cast<V *>(row + pl.at(k, 0)) + i, reinterpret_cast<const V *>(e.v)[i]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (pl.at(k, j) < D) row[pl.at(k, j)] = e.v[j];
  }
}

template <typename T, bool Q8, bool VEC, int L>
__device__ __forceinline__ void load_source(Source<T, Q8, VEC> &s, const void *base, int64_t at, const float *scales, const Place<VEC, L> &pl,
                                            int k, int D, bool on) {
  using E = typename std::conditional<Q8, int8_t, T>::type;
  load_eight<E, VEC, L>(s.e, static_cast<const E *>(base) + at, pl, k, D, on);
  if constexpr (Q8) {
#pragma unroll
    for (int i = 0; i < (VEC ? 1 : 2); ++i) s.scale[i] = on && pl.at(k, 4 * i) < D ? scales[pl.at(k, 4 * i) / kBlock] : 0.f;
  }
}

// Sums over the group's threads.  `turn` alternates the CTA-wide buffers, so that one barrier per sum is
// enough (a warp writes a buffer again only after the barrier of the sum between).
template <int L>
__device__ __forceinline__ float group_sum(float v, float (*red)[32], int &turn) {
  constexpr int kLanes = L > 0 ? L : 32;
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if constexpr (L == 0) {
    float *buf = red[turn & 1];
    ++turn;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = (int)blockDim.x >> 5;
    v = (int)(threadIdx.x & 31) < warps ? buf[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  }
  return v;
}

// The two sums at once.
template <int L>
__device__ __forceinline__ float2 group_sum2(float2 v, float2 (*red)[32], int &turn) {
  constexpr int kLanes = L > 0 ? L : 32;
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, s), __shfl_xor_sync(0xffffffffu, v.y, s)));
  if constexpr (L == 0) {
    float2 *buf = red[turn & 1];
    ++turn;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = (int)blockDim.x >> 5;
    v = (int)(threadIdx.x & 31) < warps ? buf[threadIdx.x & 31] : both(0.f);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
      v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, s), __shfl_xor_sync(0xffffffffu, v.y, s)));
  }
  return v;
}

// Absolute values' largest bits: of 16-bit types as 16-bit patterns, two at a time.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t top, const Eight<T> &e, int word) {
  if constexpr (sizeof(T) == 4) {
    return max(top, abs_bits(e.v[word]));
  } else {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(e.word(word) & 0x7fff7fffu));
    return r;
  }
}
template <typename T>
__device__ __forceinline__ uint32_t top_one(uint32_t top) {
  if constexpr (sizeof(T) == 4) return top;
  else return max(top & 0xffffu, top >> 16);
}
template <typename T>
__device__ __forceinline__ uint32_t top_as_f32(uint32_t top) {
  if constexpr (sizeof(T) == 4) return top;
  else return __float_as_uint(widen<T>(top).x);
}
// Codes of two pairs in a word: v k + 1.5 2^23 in one rounding leaves the integer in the low byte.
__device__ __forceinline__ uint32_t code_word(float2 a, float2 b, float inv) {
  a = fma2(a, both(inv), both(12582912.f));
  b = fma2(b, both(inv), both(12582912.f));
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}
// 8-bit codes of the eight values of a chunk (v: the same as fp32 pairs), and the scale of their
// block(s) by its first thread.
template <typename T, bool VEC, int L>
__device__ __forceinline__ void save_eight(const Eight<T> &raw, const float2 *v, int8_t *codes, float *scales, const Place<VEC, L> &pl, int k,
                                           int D, bool on) {
  constexpr int kWords = sizeof(T) == 4 ? 8 : 4;  // of a chunk
  Eight<int8_t> e;
  if constexpr (VEC) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) top = top_bits<T>(top, raw, i);
    top = top_one<T>(top);
    constexpr int kLanes = L > 0 && L < 16 ? L : 16;
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
    top = top_as_f32<T>(top);
    const float inv = block_inverse<T>(top);
    uint2 w;
    w.x = code_word(v[0], v[1], inv);
    w.y = code_word(v[2], v[3], inv);
    *reinterpret_cast<uint2 *>(e.v) = w;
    if (on && pl.id % 16 == 0 && pl.at(k, 0) < D) scales[pl.at(k, 0) / kBlock] = block_scale(top, inv);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kWords / 2; ++j) top = top_bits<T>(top, raw, i * kWords / 2 + j);
      top = top_as_f32<T>(__reduce_max_sync(0xffffffffu, top_one<T>(top)));
      const float inv = block_inverse<T>(top);
      reinterpret_cast<uint32_t *>(e.v)[i] = code_word(v[2 * i], v[2 * i + 1], inv);
      if (on && (threadIdx.x & 31) == 0 && pl.at(k, 4 * i) < D) scales[pl.at(k, 4 * i) / kBlock] = block_scale(top, inv);
    }
  }
  if (on) store_eight<int8_t, VEC, L>(codes, e, pl, k, D);
}

// The rows of a group: one head, tokens `first`, `first + step`, ...
struct RowWalk {
  int64_t h, t, step, part;  // part: index among the groups of this head
  bool any;                  // the group has a head
  __device__ __forceinline__ RowWalk(const NormProblem &p, int per_cta, int L) {
    const int64_t gid = (int64_t)blockIdx.x * per_cta + (L > 0 ? threadIdx.x / L : 0);
    h = gid % p.heads;
    part = t = gid / p.heads;
    step = p.groups / p.heads;
    any = h < p.H;
  }
};

// The group's weights (or biases) at pair i of the thread's channels.
template <bool VEC, int L>
__device__ __forceinline__ float2 load_columns(const float *from, const RowWalk &rw, const NormProblem &p, const Place<VEC, L> &pl, int i) {
  const int d0 = pl.at(i / 4, i % 4 * 2), d1 = pl.at(i / 4, i % 4 * 2 + 1);
  from += p.per_head && rw.any ? rw.h * p.D : 0;
  return make_float2(d0 < p.D ? from[d0] : 0.f, d1 < p.D ? from[d1] : 0.f);
}
// v - m, zero past the row's end.
template <bool VEC, int L>
__device__ __forceinline__ float2 off_mean(float2 v, float m, const Place<VEC, L> &pl, int i, int D) {
  v = add2(v, both(-m));
  return make_float2(pl.at(i / 4, i % 4 * 2) < D ? v.x : 0.f, pl.at(i / 4, i % 4 * 2 + 1) < D ? v.y : 0.f);
}
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 t = mul2(x, both(-kLog2e)), d = add2(make_float2(ex2(t.x), ex2(t.y)), both(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}
// sigmoid(x) and 1 - sigmoid(x) = e^-x sigmoid(x), each to its own relative precision; the exponent is
// held to 2^115, where the first is 0 next to any other term and the product is still 1.
__device__ __forceinline__ void sigmoid_halves(float2 x, float2 *q, float2 *rest) {
  float2 t = mul2(x, both(-kLog2e));
  asm("min.NaN.f32 %0, %0, 0f42E60000;" : "+f"(t.x));
  asm("min.NaN.f32 %0, %0, 0f42E60000;" : "+f"(t.y));
  const float2 e = make_float2(ex2(t.x), ex2(t.y)), d = add2(e, both(1.f));
  *q = make_float2(rcp(d.x), rcp(d.y));
  *rest = mul2(e, *q);
}
__device__ __forceinline__ float one_of(const float2 *v, int i) { return i & 1 ? v[i >> 1].y : v[i >> 1].x; }

template <typename T, bool VEC, int L, int K>
__global__ void __launch_bounds__(kNormThreads<L>, K == 1 && L > 0 ? FWDB : 1) gdp_norm_fwd_kernel(const NormProblem p) {
  __shared__ float red[2][32];
  int turn = 0;
  const Place<VEC, L> pl;
  const int D = (int)p.D;
  RowWalk rw(p, L > 0 ? (int)blockDim.x / (L > 0 ? L : 1) : 1, L);
  // the tokens of the warp's (or CTA's) first group: all its threads take part while that one has rows
  int64_t lead = L > 0 ? ((int64_t)blockIdx.x * blockDim.x + (threadIdx.x & ~31u)) / (L > 0 ? L : 1) / p.heads : rw.t;
  const int64_t blocks = (p.D + kBlock - 1) / kBlock;
  float2 w[4 * K], b[4 * K];
#pragma unroll
  for (int i = 0; i < 4 * K; ++i) {
    w[i] = load_columns<VEC, L>(p.w, rw, p, pl, i);
    b[i] = p.b ? load_columns<VEC, L>(p.b, rw, p, pl, i) : both(0.f);
  }
  Eight<T> o[K], z[K];
  auto load = [&](int64_t t) {
    const bool on = rw.any && t < p.T;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load_eight<T, VEC, L>(o[k], static_cast<const T *>(p.o) + t * p.o_st + rw.h * p.o_sh, pl, k, D, on);
      if (p.z) load_eight<T, VEC, L>(z[k], static_cast<const T *>(p.z) + t * p.z_st + rw.h * p.z_sh, pl, k, D, on);
    }
  };
  load(rw.t);
  int64_t row = rw.t * p.H + rw.h;
  for (; lead < p.T; lead += rw.step, rw.t += rw.step, row += rw.step * p.H) {
    const bool on = rw.any && rw.t < p.T;
    float2 v[4 * K], g[4 * K];
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) v[i] = o[i / 4].pair(i % 4);
    if (p.z) {
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) g[i] = z[i / 4].pair(i % 4);
    }
    if (p.o_codes) {
#pragma unroll
      for (int k = 0; k < K; ++k) save_eight<T, VEC, L>(o[k], v + 4 * k, p.o_codes + row * p.D, p.o_scales + row * blocks, pl, k, D, on);
      if (p.z) {
#pragma unroll
        for (int k = 0; k < K; ++k) save_eight<T, VEC, L>(z[k], g + 4 * k, p.z_codes + row * p.D, p.z_scales + row * blocks, pl, k, D, on);
      }
    }
    load(rw.t + rw.step);
    float2 s = both(0.f);
    if (p.center) {
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) s = add2(s, v[i]);
      const float m = group_sum<L>(s.x + s.y, red, turn) * p.inv_d;
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) v[i] = off_mean<VEC, L>(v[i], m, pl, i, D);
      s = both(0.f);
    }
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) s = fma2(v[i], v[i], s);
    const float r = rsqrtf(group_sum<L>(s.x + s.y, red, turn) * p.inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) v[i] = fma2(mul2(v[i], both(r)), w[i], b[i]);
    if (p.z) {
      if (p.act == GDP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4 * K; ++i) v[i] = mul2(mul2(v[i], g[i]), sigmoid2(g[i]));
      } else {
#pragma unroll
        for (int i = 0; i < 4 * K; ++i) v[i] = mul2(v[i], sigmoid2(g[i]));
      }
    } else if (p.act == GDP_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) v[i] = mul2(v[i], sigmoid2(v[i]));
    }
    if (on) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Eight<T> e;
#pragma unroll
        for (int i = 0; i < 4; ++i) e.set(i, v[4 * k + i]);
        store_eight<T, VEC, L>(static_cast<T *>(p.y) + row * p.D, e, pl, k, D);
      }
    }
  }
}

template <typename T, bool Q8, bool VEC, int L, int K>
__global__ void __launch_bounds__(kNormThreads<L>, K == 1 && L > 0 ? BWDB : 1) gdp_norm_bwd_kernel(const NormProblem p) {
  __shared__ float red[2][32];
  __shared__ float2 red2[2][32];
  __shared__ float cols[L > 0 ? 2 * 8 * kNormThreads<L> : 1];
  int turn = 0, turn2 = 0;
  const Place<VEC, L> pl;
  const int D = (int)p.D;
  RowWalk rw(p, L > 0 ? (int)blockDim.x / (L > 0 ? L : 1) : 1, L);
  int64_t lead = L > 0 ? ((int64_t)blockIdx.x * blockDim.x + (threadIdx.x & ~31u)) / (L > 0 ? L : 1) / p.heads : rw.t;
  const int64_t blocks = (p.D + kBlock - 1) / kBlock;
  const bool zed = Q8 ? p.z_codes_in != nullptr : p.z != nullptr;
  float2 w[4 * K], sw[4 * K], sb[4 * K];
#pragma unroll
  for (int i = 0; i < 4 * K; ++i) {
    w[i] = load_columns<VEC, L>(p.w, rw, p, pl, i);
    sw[i] = sb[i] = both(0.f);
  }
  Source<T, Q8, VEC> o[K], z[K];
  Eight<T> y[K];
  auto load = [&](int64_t t) {
    const bool on = rw.any && t < p.T;
    const int64_t row = t * p.H + rw.h;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load_eight<T, VEC, L>(y[k], static_cast<const T *>(p.dy) + t * p.dy_st + rw.h * p.dy_sh, pl, k, D, on);
      if constexpr (Q8) {
        load_source<T, true, VEC, L>(o[k], p.o_codes_in, row * p.D, p.o_scales_in + row * blocks, pl, k, D, on);
        if (zed) load_source<T, true, VEC, L>(z[k], p.z_codes_in, row * p.D, p.z_scales_in + row * blocks, pl, k, D, on);
      } else {
        load_source<T, false, VEC, L>(o[k], p.o, t * p.o_st + rw.h * p.o_sh, nullptr, pl, k, D, on);
        if (zed) load_source<T, false, VEC, L>(z[k], p.z, t * p.z_st + rw.h * p.z_sh, nullptr, pl, k, D, on);
      }
    }
  };
  load(rw.t);
  int64_t row = rw.t * p.H + rw.h;
  for (; lead < p.T; lead += rw.step, rw.t += rw.step, row += rw.step * p.H) {
    const bool on = rw.any && rw.t < p.T;
    float2 n[4 * K], g[4 * K], dn[4 * K];
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) {
      n[i] = o[i / 4].pair(i % 4);
      dn[i] = y[i / 4].pair(i % 4);
    }
    if (zed) {
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) g[i] = z[i / 4].pair(i % 4);
    }
    load(rw.t + rw.step);
    float2 s = both(0.f);
    if (p.center) {
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) s = add2(s, n[i]);
      const float m = group_sum<L>(s.x + s.y, red, turn) * p.inv_d;
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) n[i] = off_mean<VEC, L>(n[i], m, pl, i, D);
      s = both(0.f);
    }
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) s = fma2(n[i], n[i], s);
    float r = rsqrtf(group_sum<L>(s.x + s.y, red, turn) * p.inv_d + p.eps);
    if (!on) r = 0.f;  // a group without a row adds zeros to its sums
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) n[i] = mul2(n[i], both(r));
    // through the activation: dn from dy to du = dL/du, g from z to dz
    auto gate = [&](auto zed_, auto silu_) {
      constexpr bool kZed = decltype(zed_)::value, kSilu = decltype(silu_)::value;
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) {
        float2 u = mul2(n[i], w[i]);
        if (p.b) u = add2(u, load_columns<VEC, L>(p.b, rw, p, pl, i));
        const float2 x = kZed ? g[i] : u;
        float2 q, rest;
        sigmoid_halves(x, &q, &rest);
        const float2 slope = kSilu ? mul2(q, fma2(x, rest, both(1.f))) : mul2(q, rest);
        if (kZed) {
          g[i] = mul2(mul2(dn[i], u), slope);
          dn[i] = mul2(dn[i], kSilu ? mul2(x, q) : q);
        } else {
          dn[i] = mul2(dn[i], slope);
        }
      }
    };
    if (zed) {
      if (p.act == GDP_ACT_SILU) gate(std::true_type{}, std::true_type{});
      else gate(std::true_type{}, std::false_type{});
      if (on) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          Eight<T> e;
#pragma unroll
          for (int i = 0; i < 4; ++i) e.set(i, g[4 * k + i]);
          store_eight<T, VEC, L>(static_cast<T *>(p.d_z) + row * p.D, e, pl, k, D);
        }
      }
    } else if (p.act == GDP_ACT_SILU) {
      gate(std::false_type{}, std::true_type{});
    }
    float2 s1 = both(0.f), s2 = both(0.f);
    if (p.b) {
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) sb[i] = add2(sb[i], dn[i]);
    }
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) {
      sw[i] = fma2(dn[i], n[i], sw[i]);
      dn[i] = mul2(dn[i], w[i]);
      s2 = fma2(dn[i], n[i], s2);
    }
    float m1 = 0.f, m2;
    if (p.center) {
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) s1 = add2(s1, dn[i]);
      const float2 t = group_sum2<L>(make_float2(s1.x + s1.y, s2.x + s2.y), red2, turn2);
      m1 = t.x * p.inv_d;
      m2 = t.y * p.inv_d;
    } else {
      m2 = group_sum<L>(s2.x + s2.y, red, turn) * p.inv_d;
    }
    if (on) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Eight<T> e;
#pragma unroll
        for (int i = 0; i < 4; ++i) e.set(i, mul2(fma2(n[4 * k + i], both(-m2), add2(dn[4 * k + i], both(-m1))), both(r)));
        store_eight<T, VEC, L>(static_cast<T *>(p.d_o) + row * p.D, e, pl, k, D);
      }
    }
  }
  // column sums: [part][columns], all dweight parts before all dbias parts
  const int64_t ncols = p.per_head ? p.H * p.D : p.D;
  if (L == 0 || p.per_head) {
    const int64_t part = p.per_head ? rw.part : blockIdx.x, off = p.per_head ? rw.h * p.D : 0;
#pragma unroll
    for (int i = 0; i < 8 * K; ++i) {
      const int d = pl.at(i / 8, i % 8);
      if (rw.any && d < D) {
        p.partial[part * ncols + off + d] = one_of(sw, i);
        if (p.b) p.partial[(p.parts + part) * ncols + off + d] = one_of(sb, i);
      }
    }
  } else if constexpr (L > 0) {  // one part per CTA: the groups' sums in turn
    constexpr int kGroups = kNormThreads<L> / L;
    const int group = (int)threadIdx.x / L;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cols[group * 8 * L + pl.at(0, j)] = rw.any ? one_of(sw, j) : 0.f;
      cols[(kGroups + group) * 8 * L + pl.at(0, j)] = rw.any ? one_of(sb, j) : 0.f;
    }
    __syncthreads();
    for (int d = (int)threadIdx.x; d < 2 * D; d += (int)blockDim.x) {
      const int which = d >= D, c = d - which * D;
      if (which && !p.b) break;
      float s = 0.f;
#pragma unroll 4
      for (int i = 0; i < kGroups; ++i) s += cols[(which * kGroups + i) * 8 * L + c];
      p.partial[(which * p.parts + blockIdx.x) * ncols + c] = s;
    }
  }
}

template <typename T, bool VEC, int L, int K>
cudaError_t run_norm_fwd(const NormProblem &p, const NormPlan &n, cudaStream_t stream) {
  gdp_norm_fwd_kernel<T, VEC, L, K><<<(unsigned)n.grid, n.threads, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, bool VEC, int L, int K>
cudaError_t run_norm_bwd(const NormProblem &p, const NormPlan &n, cudaStream_t stream) {
  if (p.o_codes_in) gdp_norm_bwd_kernel<T, true, VEC, L, K><<<(unsigned)n.grid, n.threads, 0, stream>>>(p);
  else gdp_norm_bwd_kernel<T, false, VEC, L, K><<<(unsigned)n.grid, n.threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

#define GDP_NORM_CASES(RUN)                                              \
  if (n.vec) {                                                           \
    if (n.lanes == 8) return RUN<T, true, 8, 1>(p, n, stream);           \
    if (n.lanes == 16) return RUN<T, true, 16, 1>(p, n, stream);         \
    if (n.lanes == 32) return RUN<T, true, 32, 1>(p, n, stream);         \
    if (n.chunks == 1) return RUN<T, true, 0, 1>(p, n, stream);          \
    return RUN<T, true, 0, 2>(p, n, stream);                             \
  }                                                                      \
  if (n.lanes == 32) return RUN<T, false, 32, 1>(p, n, stream);          \
  if (n.chunks == 1) return RUN<T, false, 0, 1>(p, n, stream);           \
  return RUN<T, false, 0, 2>(p, n, stream);

template <typename T>
cudaError_t launch_norm_fwd(const NormProblem &p, const NormPlan &n, cudaStream_t stream) {
  GDP_NORM_CASES(run_norm_fwd)
}
template <typename T>
cudaError_t launch_norm_bwd(const NormProblem &p, const NormPlan &n, cudaStream_t stream) {
  GDP_NORM_CASES(run_norm_bwd)
}
#undef GDP_NORM_CASES

}  // namespace layer
}  // namespace gdp
