// gdp_norm_body.cuh -- the grouped norm with an activated gate: forward (with 8-bit checkpoints) and
// backward kernels (gdp_layer.h).
//
// A row (token, head) is held by a group of threads, sixteen channels per thread: 4, 8, 16 or 32 lanes
// of a warp (D up to 64, 128, 256, 512), or a whole CTA.  A group keeps one head, so that the backward's
// sums over tokens (dweight, dbias) accumulate in registers; it walks over tokens with the next row's
// loads in flight.  Those sums leave once per CTA (or per group where every head has its own weights)
// and a second kernel adds them up in a fixed order.
//
// Bound: 65536 x 32 x 128 bf16 with a gate takes 337 us forward with checkpoints (2.16 GB, 6.4 TB/s: memory) and
// about 435 us backward from them (2.16 GB, 5.0 TB/s).  The backward takes 35 instructions per channel, issues on
// 55 % of the cycles and draws 54 % of the memory's peak: 128 registers hold the row, its gradient and the
// column sums, and two CTAs per SM (16 warps) do not hide the loads.  More warps spill (three CTAs 1244 against 834 us for
// the training step), and with dweight's sums in shared memory too (1057 and, two CTAs, 807 against 783 us).
#pragma once

#include "gdp_norm.cuh"

namespace gdp {
namespace layer {
namespace {

constexpr int kPer = 16;  // channels of a thread: 8 cost 42 instructions per channel in the reductions and
                          // addresses alone (966 us for the training step of 65536 x 32 x 128)

// Wide rows' forward CTAs have at most 512 threads; the larger bound holds the compiler to 80 registers, so
// that three of 256 threads share an SM (1421 x 4096: 13.1 us, with 114 registers 14.9 us).
constexpr int kWideFwdBound = 768;

// Where a thread's channels lie in its row.  VEC: sixteen consecutive ones; else strided by the width of
// a run of lanes, so that the lanes' accesses are runs of memory.  Either way a checkpoint block of 128
// channels lies in eight lanes (a shorter row in its four).
template <bool VEC, int L>
struct Place {
  static constexpr int kRun = L == 4 ? 4 : 8;
  int id, first;     // thread of the group, its first channel
  bool in[2];        // VEC: its two halves lie in the row
  __device__ __forceinline__ explicit Place(int D) {
    id = L > 0 ? (int)threadIdx.x % (L > 0 ? L : 1) : (int)threadIdx.x;
    first = VEC ? id * kPer : id / kRun * (kRun * kPer) + id % kRun;
    in[0] = first < D;
    in[1] = first + 8 < D;
  }
  __device__ __forceinline__ int at(int j) const { return first + (VEC ? j : kRun * j); }
  __device__ __forceinline__ bool leads_block() const { return id % kRun == 0; }
  __device__ __forceinline__ int block() const { return first / kBlock; }
};

// Sixteen values of a row as they lie in memory.
template <typename T>
struct alignas(16) Sixteen {
  T v[kPer];
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

// Loads and stores of a row, `at` pointing to the thread's first channel.  VEC: 16 bytes at a time, eight
// channels (of codes: eight or sixteen), D a multiple of eight.
template <typename T, bool VEC, int L>
__device__ __forceinline__ void load_row(Sixteen<T> &e, const T *at, const Place<VEC, L> &pl, int D, bool on) {
  if constexpr (VEC && sizeof(T) == 1) {
    uint2 *to = reinterpret_cast<uint2 *>(e.v);
    const uint2 *from = reinterpret_cast<const uint2 *>(at);
    to[0] = on && pl.in[0] ? __ldcs(from) : make_uint2(0u, 0u);
    to[1] = on && pl.in[1] ? __ldcs(from + 1) : make_uint2(0u, 0u);
  } else if constexpr (VEC) {
    uint4 *to = reinterpret_cast<uint4 *>(e.v);
    const uint4 *from = reinterpret_cast<const uint4 *>(at);
    constexpr int n = (int)sizeof(T);  // 16-byte words
#pragma unroll
    for (int i = 0; i < n; ++i) to[i] = on && pl.in[i / (n / 2)] ? __ldcs(from + i) : make_uint4(0u, 0u, 0u, 0u);
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool in = on && pl.at(j) < D;
      if constexpr (sizeof(T) == 1) e.v[j] = in ? at[pl.kRun * j] : (T)0;
      else e.v[j] = in ? at[pl.kRun * j] : from_f32<T>(0.f);
    }
  }
}
template <typename T, bool VEC, int L>
__device__ __forceinline__ void store_row(T *at, const Sixteen<T> &e, const Place<VEC, L> &pl, int D, bool on) {
  if constexpr (VEC && sizeof(T) == 1) {
    const uint2 *from = reinterpret_cast<const uint2 *>(e.v);
    uint2 *to = reinterpret_cast<uint2 *>(at);
    if (on && pl.in[0]) __stcs(to, from[0]);
    if (on && pl.in[1]) __stcs(to + 1, from[1]);
  } else if constexpr (VEC) {
    const uint4 *from = reinterpret_cast<const uint4 *>(e.v);
    uint4 *to = reinterpret_cast<uint4 *>(at);
    constexpr int n = (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (on && pl.in[i / (n / 2)]) __stcs(to + i, from[i]);
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (on && pl.at(j) < D) at[pl.kRun * j] = e.v[j];
  }
}

// Source of the backward's o and z: a tensor, or codes with the scale of the block they lie in.
template <typename T, bool Q8>
struct Source {
  Sixteen<typename std::conditional<Q8, int8_t, T>::type> e;
  float scale;
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (Q8) {
      // a byte plus 128 under the exponent of 2^23 is 2^23 + 128 + code
      const uint32_t w = e.word(i >> 1) ^ 0x80808080u;
      const float2 m = make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + (i & 1) * 2)),
                                   __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441 + (i & 1) * 2)));
      return mul2(add2(m, both(-8388736.f)), both(scale));
    } else {
      return e.pair(i);
    }
  }
};
template <typename T, bool Q8, bool VEC, int L>
__device__ __forceinline__ void load_source(Source<T, Q8> &s, const void *tensor, const int8_t *codes, const float *scales, int64_t at,
                                            int64_t scale_at, const Place<VEC, L> &pl, int D, bool on) {
  if constexpr (Q8) {
    load_row<int8_t, VEC, L>(s.e, codes + at, pl, D, on);
    s.scale = on && pl.in[0] ? __ldcs(scales + scale_at) : 0.f;
  } else {
    load_row<T, VEC, L>(s.e, static_cast<const T *>(tensor) + at, pl, D, on);
  }
}

// The group's weights (or biases) at pairs i and i + 1 of the thread's channels: read for every row (a few
// KB that stay in L1), so that they take no registers meanwhile.
template <bool VEC, int L>
__device__ __forceinline__ void load_columns(float2 *to, const float *from, int i, const Place<VEC, L> &pl, int D, int vec) {
  if (VEC && vec) {
    const float4 q = pl.in[i / 4] ? __ldg(reinterpret_cast<const float4 *>(from) + i / 2) : make_float4(0.f, 0.f, 0.f, 0.f);
    to[0] = make_float2(q.x, q.y);
    to[1] = make_float2(q.z, q.w);
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int d0 = pl.at(2 * (i + u)), d1 = pl.at(2 * (i + u) + 1);
      to[u] = make_float2(d0 < D ? __ldg(from + d0 - pl.first) : 0.f, d1 < D ? __ldg(from + d1 - pl.first) : 0.f);
    }
  }
}

// Sums over the group's threads, one or two at once.  `turn` alternates the CTA-wide buffers, so that one
// barrier per sum is enough (a warp writes a buffer again only after the barrier of the sum between).
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return add2(a, b); }
__device__ __forceinline__ float from_lane(float v, int s) { return __shfl_xor_sync(0xffffffffu, v, s); }
__device__ __forceinline__ float2 from_lane(float2 v, int s) { return make_float2(from_lane(v.x, s), from_lane(v.y, s)); }
template <int L, typename V>
__device__ __forceinline__ V group_sum(V v, float2 (*red)[32], int &turn) {
  constexpr int kLanes = L > 0 ? L : 32;
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1) v = plus(v, from_lane(v, s));
  if constexpr (L == 0) {
    // up to 16 warps' values: single sums in the first 64 bytes, pairs in the 128 after them
    V *buf = reinterpret_cast<V *>(red[turn & 1] + (sizeof(V) == 4 ? 0 : 8));
    ++turn;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    // the warps' sums, 16 bytes at a time (the buffers' unused ends are zero)
    const int warps = (int)blockDim.x >> 5;
    constexpr int kEach = 16 / (int)sizeof(V);
    float4 sum = *reinterpret_cast<const float4 *>(buf);
    for (int i = kEach; i < warps; i += kEach) {
      const float4 q = *reinterpret_cast<const float4 *>(buf + i);
      sum = make_float4(sum.x + q.x, sum.y + q.y, sum.z + q.z, sum.w + q.w);
    }
    if constexpr (sizeof(V) == 4) v = (sum.x + sum.y) + (sum.z + sum.w);
    else v = make_float2(sum.x + sum.z, sum.y + sum.w);
  }
  return v;
}

// ---- checkpoints ----
// Largest absolute value of the sixteen: bits of the type itself (NaN above all).
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const Sixteen<T> &e) {
  uint32_t top = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = max(top, abs_bits(e.v[i]));
    return top;
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    T2 m = __habs2(*reinterpret_cast<const T2 *>(&e.v[0]));
#pragma unroll
    for (int i = 1; i < kPer / 2; ++i) m = __hmax2_nan(__habs2(*reinterpret_cast<const T2 *>(&e.v[2 * i])), m);
    top = *reinterpret_cast<const uint32_t *>(&m);
    return max(top & 0xffffu, top >> 16);
  }
}
// Of the block: two tensors' at once.
template <typename T, int L>
__device__ __forceinline__ void block_tops(uint32_t &a, uint32_t &b) {
  constexpr int kRun = L == 4 ? 4 : 8;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int s = kRun / 2; s > 0; s >>= 1) {
      a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
      b = max(b, __shfl_xor_sync(0xffffffffu, b, s));
    }
  } else {
    uint32_t t = a | b << 16;
#pragma unroll
    for (int s = kRun / 2; s > 0; s >>= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, s));
    a = __float_as_uint(widen<T>(t).x);
    b = __float_as_uint(widen<T>(t).y);
  }
}
// Codes of two pairs in a word: v k + 1.5 2^23 leaves the integer in the low byte.  The product is exact for
// 16-bit types and rounded to fp32 first for fp32 values, so that the codes are those of plain fp32 arithmetic.
template <typename T>
__device__ __forceinline__ float2 code_pair(float2 v, float inv) {
  // (one by one: the paired operations came out contracted)
  if constexpr (sizeof(T) == 4) return make_float2(__fadd_rn(__fmul_rn(v.x, inv), 12582912.f), __fadd_rn(__fmul_rn(v.y, inv), 12582912.f));
  else return fma2(v, both(inv), both(12582912.f));
}
template <typename T>
__device__ __forceinline__ uint32_t code_word(float2 a, float2 b, float inv) {
  a = code_pair<T>(a, inv);
  b = code_pair<T>(b, inv);
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}
template <typename T, bool VEC, int L>
__device__ __forceinline__ void save_row(const Sixteen<T> &v, uint32_t top, int8_t *codes, float *scale, const Place<VEC, L> &pl, int D, bool on) {
  const float inv = block_inverse<T>(top);
  Sixteen<int8_t> e;
#pragma unroll
  for (int i = 0; i < kPer / 4; ++i) reinterpret_cast<uint32_t *>(e.v)[i] = code_word<T>(v.pair(2 * i), v.pair(2 * i + 1), inv);
  store_row<int8_t, VEC, L>(codes, e, pl, D, on);
  if (on && pl.leads_block() && pl.in[0]) *scale = block_scale(top, inv);
}

// ---- arithmetic of a row ----
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 t = mul2(x, both(-kLog2e)), d = add2(make_float2(ex2(t.x), ex2(t.y)), both(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}
// v less its mean where centred (zero past the row's end), and the reciprocal root of its mean square.
template <bool VEC, int L>
__device__ __forceinline__ float row_stats(float2 *v, const NormProblem &p, const Place<VEC, L> &pl, int D, float2 (*red)[32], int &turn) {
  constexpr int P = kPer / 2;
  if (p.center) {
    float2 s = v[0];
#pragma unroll
    for (int i = 1; i < P; ++i) s = add2(s, v[i]);
    const float m = group_sum<L>(s.x + s.y, red, turn) * p.inv_d;
    const bool whole = VEC ? pl.in[1] : pl.at(kPer - 1) < D;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[i] = add2(v[i], both(-m));
      if (!whole) v[i] = make_float2(pl.at(2 * i) < D ? v[i].x : 0.f, pl.at(2 * i + 1) < D ? v[i].y : 0.f);
    }
  }
  float2 s = mul2(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < P; ++i) s = fma2(v[i], v[i], s);
  return rsqrtf(group_sum<L>(s.x + s.y, red, turn) * p.inv_d + p.eps);
}

// The rows of a group: one head, tokens t, t + step, ...
struct RowWalk {
  uint32_t t, step;  // T is below 2^31, so that neither passes 2^32
  uint32_t lead;     // token of the warp's (or CTA's) first group: its threads go on together while that one has rows
  int h;
  bool any;          // the group has a head
  __device__ __forceinline__ RowWalk(const NormProblem &p, int L) {
    const int64_t per_cta = L > 0 ? blockDim.x / L : 1, gid = blockIdx.x * per_cta + (L > 0 ? threadIdx.x / L : 0);
    h = (int)(gid % p.heads);
    t = (uint32_t)(gid / p.heads);  // also the group's index among those of its head
    step = (uint32_t)(p.groups / p.heads);
    any = h < p.H;
    lead = L > 0 ? (uint32_t)((blockIdx.x * per_cta + (threadIdx.x & ~31u) / L) / p.heads) : t;
  }
};

template <typename T, bool VEC, int L>
__global__ void __launch_bounds__(L > 0 ? kNormThreads<L> : kWideFwdBound, L > 0 ? kNormFwdCtas : 1) gdp_norm_fwd_kernel(const NormProblem p) {
  constexpr int P = kPer / 2;
  __shared__ __align__(16) float2 red[2][32];
  int turn = 0;
  if (L == 0) {
    if (threadIdx.x < 64) red[threadIdx.x >> 5][threadIdx.x & 31] = both(0.f);
    __syncthreads();
  }
  const int D = (int)p.D, blocks = (D + kBlock - 1) / kBlock;
  const Place<VEC, L> pl(D);
  RowWalk rw(p, L);
  const int64_t col = (p.per_head && rw.any ? (int64_t)rw.h * D : 0) + pl.first;
  const float *w = p.w + col, *b = p.b ? p.b + col : nullptr;
  const bool zed = p.z != nullptr, save = p.o_codes != nullptr;
  int64_t o_at = (int64_t)rw.t * p.o_st + rw.h * p.o_sh + pl.first, z_at = (int64_t)rw.t * p.z_st + rw.h * p.z_sh + pl.first;
  Sixteen<T> next_o, next_z;
  auto load = [&](bool on) {
    load_row<T, VEC, L>(next_o, static_cast<const T *>(p.o) + o_at, pl, D, on);
    if (zed) load_row<T, VEC, L>(next_z, static_cast<const T *>(p.z) + z_at, pl, D, on);
    o_at += rw.step * p.o_st;
    z_at += rw.step * p.z_st;
  };
  load(rw.any && rw.t < p.T);
  // offset of the thread's channels, and of their block's scale, in the outputs
  int64_t at = ((int64_t)rw.t * p.H + rw.h) * D + pl.first, scale_at = ((int64_t)rw.t * p.H + rw.h) * blocks + pl.block();
  const int64_t step = rw.step * p.H * D, scale_step = rw.step * p.H * blocks;
  for (; rw.lead < p.T; rw.lead += rw.step, rw.t += rw.step, at += step, scale_at += scale_step) {
    const bool on = rw.any && rw.t < p.T;
    Sixteen<T> e = next_o;
    const Sixteen<T> z = next_z;
    load(rw.any && rw.t + rw.step < p.T);
    if (save) {
      uint32_t a = top_bits<T>(e), c = zed ? top_bits<T>(z) : 0u;
      block_tops<T, L>(a, c);
      save_row<T, VEC, L>(e, a, p.o_codes + at, p.o_scales + scale_at, pl, D, on);
      if (zed) save_row<T, VEC, L>(z, c, p.z_codes + at, p.z_scales + scale_at, pl, D, on);
    }
    float2 v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = e.pair(i);
    const float r = row_stats<VEC, L>(v, p, pl, D, red, turn);
    auto finish = [&](auto zed_, auto act_) {
      constexpr bool kZed = decltype(zed_)::value;
      constexpr int kAct = decltype(act_)::value;
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        float2 cw[2], cb[2] = {both(0.f), both(0.f)};
        load_columns<VEC, L>(cw, w, i, pl, D, p.vec_cols);
        if (b) load_columns<VEC, L>(cb, b, i, pl, D, p.vec_cols);
#pragma unroll
        for (int u = i; u < i + 2; ++u) {
          float2 x = fma2(mul2(v[u], both(r)), cw[u - i], cb[u - i]);
          if constexpr (kZed) {
            const float2 g = z.pair(u);
            // g sigmoid(g) first: for g next to the type's lowest value it is 0, while x g overflows
            x = mul2(x, kAct == GDP_ACT_SILU ? mul2(g, sigmoid2(g)) : sigmoid2(g));
          } else if constexpr (kAct == GDP_ACT_SILU) {
            x = mul2(x, sigmoid2(x));
          }
          e.set(u, x);
        }
      }
    };
    using Silu = std::integral_constant<int, GDP_ACT_SILU>;
    if (zed) {
      if (p.act == GDP_ACT_SILU) finish(std::true_type{}, Silu{});
      else finish(std::true_type{}, std::integral_constant<int, GDP_ACT_SIGMOID>{});
    } else if (p.act == GDP_ACT_SILU) {
      finish(std::false_type{}, Silu{});
    } else {
      finish(std::false_type{}, std::integral_constant<int, GDP_ACT_NONE>{});
    }
    store_row<T, VEC, L>(static_cast<T *>(p.y) + at, e, pl, D, on);
  }
}

template <typename T, bool Q8, bool VEC, int L>
__global__ void __launch_bounds__(kNormThreads<L>, L > 0 ? kNormBwdCtas : 1) gdp_norm_bwd_kernel(const NormProblem p) {
  constexpr int P = kPer / 2;
  __shared__ __align__(16) float2 red[2][32];
  int turn = 0;
  if (L == 0) {
    if (threadIdx.x < 64) red[threadIdx.x >> 5][threadIdx.x & 31] = both(0.f);
    __syncthreads();
  }
  const int D = (int)p.D, blocks = (D + kBlock - 1) / kBlock;
  const Place<VEC, L> pl(D);
  RowWalk rw(p, L);
  const bool zed = Q8 ? p.z_codes_in != nullptr : p.z != nullptr;
  const int64_t col = (p.per_head && rw.any ? (int64_t)rw.h * D : 0) + pl.first;
  const float *w = p.w + col, *b = p.b ? p.b + col : nullptr;
  // sums over tokens: dweight's in registers, dbias's (fewer calls have one) in shared memory
  __shared__ float4 side[kPer / 4][kNormThreads<L>];
  float2 sw[P];
#pragma unroll
  for (int i = 0; i < P; ++i) sw[i] = both(0.f);
  if (b) {
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) side[i][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // offsets of the thread's channels: in the outputs and the codes (and of their block's scale), and of the
  // next row in the strided tensors
  int64_t at = ((int64_t)rw.t * p.H + rw.h) * D + pl.first, scale_at = ((int64_t)rw.t * p.H + rw.h) * blocks + pl.block();
  int64_t y_at = (int64_t)rw.t * p.dy_st + rw.h * p.dy_sh + pl.first;
  int64_t o_at = (int64_t)rw.t * p.o_st + rw.h * p.o_sh + pl.first, z_at = (int64_t)rw.t * p.z_st + rw.h * p.z_sh + pl.first;
  const int64_t step = rw.step * p.H * D;
  Source<T, Q8> next_o, next_z;
  Sixteen<T> next_y;
  auto load = [&](int64_t codes_at, bool on) {
    load_row<T, VEC, L>(next_y, static_cast<const T *>(p.dy) + y_at, pl, D, on);
    load_source<T, Q8, VEC, L>(next_o, p.o, p.o_codes_in, p.o_scales_in, Q8 ? codes_at : o_at, scale_at, pl, D, on);
    if (zed) load_source<T, Q8, VEC, L>(next_z, p.z, p.z_codes_in, p.z_scales_in, Q8 ? codes_at : z_at, scale_at, pl, D, on);
    y_at += rw.step * p.dy_st;
    if constexpr (Q8) {
      scale_at += rw.step * p.H * blocks;
    } else {
      o_at += rw.step * p.o_st;
      z_at += rw.step * p.z_st;
    }
  };
  load(at, rw.any && rw.t < p.T);
  for (; rw.lead < p.T; rw.lead += rw.step, rw.t += rw.step, at += step) {
    const bool on = rw.any && rw.t < p.T;
    const Source<T, Q8> z = next_z;
    Sixteen<T> e = next_y;  // dy, then dz in its place
    float2 n[P], dn[P];
#pragma unroll
    for (int i = 0; i < P; ++i) n[i] = next_o.pair(i);
    load(at + step, rw.any && rw.t + rw.step < p.T);
    float r = row_stats<VEC, L>(n, p, pl, D, red, turn);
    if (!on) r = 0.f;  // a group without a row adds zeros to its sums
    float2 s1 = both(0.f), s2 = both(0.f);
    // through the activation: du = dL/du and dz; then dn = du w
    auto gate = [&](auto zed_, auto act_) {
      constexpr bool kZed = decltype(zed_)::value;
      constexpr int kAct = decltype(act_)::value;
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        float2 cw[2], cb[2] = {both(0.f), both(0.f)}, du[2];
        load_columns<VEC, L>(cw, w, i, pl, D, p.vec_cols);
        if (b && kAct != GDP_ACT_NONE) load_columns<VEC, L>(cb, b, i, pl, D, p.vec_cols);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          n[i + k] = mul2(n[i + k], both(r));
          du[k] = e.pair(i + k);
          if constexpr (kAct != GDP_ACT_NONE) {
            const float2 u = fma2(n[i + k], cw[k], cb[k]), x = kZed ? z.pair(i + k) : u;
            float2 q, rest;
            sigmoid_halves(x, &q, &rest);
            const float2 slope = kAct == GDP_ACT_SILU ? mul2(q, fma2(x, rest, both(1.f))) : mul2(q, rest);
            if constexpr (kZed) {
              e.set(i + k, mul2(mul2(du[k], u), slope));
              du[k] = mul2(du[k], kAct == GDP_ACT_SILU ? mul2(x, q) : q);
            } else {
              du[k] = mul2(du[k], slope);
            }
          }
          sw[i + k] = fma2(du[k], n[i + k], sw[i + k]);
          dn[i + k] = mul2(du[k], cw[k]);
          s1 = add2(s1, dn[i + k]);
          s2 = fma2(dn[i + k], n[i + k], s2);
        }
        if (b) {
          float4 t = side[i / 2][threadIdx.x];
          side[i / 2][threadIdx.x] = make_float4(t.x + du[0].x, t.y + du[0].y, t.z + du[1].x, t.w + du[1].y);
        }
      }
    };
    using Silu = std::integral_constant<int, GDP_ACT_SILU>;
    if (zed) {
      if (p.act == GDP_ACT_SILU) gate(std::true_type{}, Silu{});
      else gate(std::true_type{}, std::integral_constant<int, GDP_ACT_SIGMOID>{});
      store_row<T, VEC, L>(static_cast<T *>(p.d_z) + at, e, pl, D, on);
    } else if (p.act == GDP_ACT_SILU) {
      gate(std::false_type{}, Silu{});
    } else {
      gate(std::false_type{}, std::integral_constant<int, GDP_ACT_NONE>{});
    }
    const float2 t = group_sum<L>(make_float2(s1.x + s1.y, s2.x + s2.y), red, turn);
    const float m1 = p.center ? t.x * p.inv_d : 0.f, m2 = t.y * p.inv_d;
#pragma unroll
    for (int i = 0; i < P; ++i) e.set(i, mul2(fma2(n[i], both(-m2), add2(dn[i], both(-m1))), both(r)));
    store_row<T, VEC, L>(static_cast<T *>(p.d_o) + at, e, pl, D, on);
  }
  sm100::pdl_trigger();  // the kernel that adds them up may get ready
  // column sums: [part][columns], all dweight parts before all dbias parts
  const int64_t ncols = p.per_head ? p.H * p.D : p.D;
  for (int which = 0; which < (b ? 2 : 1); ++which) {
    if (which) {
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i) {
        const float4 t = side[i][threadIdx.x];
        sw[2 * i] = make_float2(t.x, t.y);
        sw[2 * i + 1] = make_float2(t.z, t.w);
      }
    }
    float *to = p.partial + which * p.parts * ncols;
    if (L == 0 || p.per_head) {
      const int64_t gid = (int64_t)blockIdx.x * (L > 0 ? blockDim.x / (L > 0 ? L : 1) : 1) + (L > 0 ? threadIdx.x / (L > 0 ? L : 1) : 0);
      to += (p.per_head ? gid / p.heads : (int64_t)blockIdx.x) * ncols + (p.per_head ? rw.h * p.D : 0);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (rw.any && pl.at(j) < D) to[pl.at(j)] = j & 1 ? sw[j >> 1].y : sw[j >> 1].x;
    } else if constexpr (L > 0) {  // one part per CTA: the groups' sums in turn
      constexpr int kGroups = kNormThreads<L> / L, kWide = kPer * L;
      __shared__ float cols[kGroups * kWide];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; ++j) cols[(int)threadIdx.x / L * kWide + pl.at(j)] = rw.any ? (j & 1 ? sw[j >> 1].y : sw[j >> 1].x) : 0.f;
      __syncthreads();
      for (int d = (int)threadIdx.x; d < D; d += (int)blockDim.x) {
        float t = 0.f;
#pragma unroll 8
        for (int i = 0; i < kGroups; ++i) t += cols[i * kWide + d];
        to[blockIdx.x * ncols + d] = t;
      }
    }
  }
}

template <typename T, bool VEC, int L>
cudaError_t run_norm_fwd(const NormProblem &p, const NormPlan &n, cudaStream_t stream) {
  gdp_norm_fwd_kernel<T, VEC, L><<<(unsigned)n.grid, n.threads, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, bool VEC, int L>
cudaError_t run_norm_bwd(const NormProblem &p, const NormPlan &n, cudaStream_t stream) {
  if (p.o_codes_in) gdp_norm_bwd_kernel<T, true, VEC, L><<<(unsigned)n.grid, n.threads, 0, stream>>>(p);
  else gdp_norm_bwd_kernel<T, false, VEC, L><<<(unsigned)n.grid, n.threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

#define GDP_NORM_CASES(RUN)                                   \
  if (n.vec) {                                                \
    if (n.lanes == 4) return RUN<T, true, 4>(p, n, stream);   \
    if (n.lanes == 8) return RUN<T, true, 8>(p, n, stream);   \
    if (n.lanes == 16) return RUN<T, true, 16>(p, n, stream); \
    if (n.lanes == 32) return RUN<T, true, 32>(p, n, stream); \
    return RUN<T, true, 0>(p, n, stream);                     \
  }                                                           \
  if (n.lanes == 8) return RUN<T, false, 8>(p, n, stream);    \
  if (n.lanes == 32) return RUN<T, false, 32>(p, n, stream);  \
  return RUN<T, false, 0>(p, n, stream);

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
