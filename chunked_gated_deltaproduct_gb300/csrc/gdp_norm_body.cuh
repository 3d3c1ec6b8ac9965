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
};
// Source of o and z: a tensor, or codes with the scales of the (one or two) blocks the eight lie in.
template <typename T, bool Q8, bool VEC>
struct Source {
  Eight<typename std::conditional<Q8, int8_t, T>::type> e;
  float scale[Q8 ? (VEC ? 1 : 2) : 1];
  __device__ __forceinline__ float get(int j) const {
    if constexpr (Q8) return (float)e.v[j] * scale[VEC ? 0 : j >> 2];
    else return to_f32(e.v[j]);
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

// 8-bit codes of the eight values of a chunk, and the scale of their block(s) by its first thread.
template <bool VEC, int L>
__device__ __forceinline__ void save_eight(const float *v, int8_t *codes, float *scales, const Place<VEC, L> &pl, int k, int D, bool on) {
  Eight<int8_t> e;
  if constexpr (VEC) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, abs_bits(v[j]));
    constexpr int kLanes = L > 0 && L < 16 ? L : 16;
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
    const float inv = block_inverse(top);
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = block_code(v[j], inv);
    uint2 w;
    w.x = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    w.y = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
    *reinterpret_cast<uint2 *>(e.v) = w;
    if (on && pl.id % 16 == 0 && pl.at(k, 0) < D) scales[pl.at(k, 0) / kBlock] = block_scale(top, inv);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, abs_bits(v[4 * i + j]));
      top = __reduce_max_sync(0xffffffffu, top);
      const float inv = block_inverse(top);
#pragma unroll
      for (int j = 0; j < 4; ++j) e.v[4 * i + j] = (int8_t)block_code(v[4 * i + j], inv);
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
  float w[8 * K], b[8 * K];
#pragma unroll
  for (int i = 0; i < 8 * K; ++i) {
    const int d = pl.at(i / 8, i % 8);
    const int64_t col = (p.per_head ? rw.h * p.D : 0) + d;
    w[i] = rw.any && d < D ? p.w[col] : 0.f;
    b[i] = p.b && rw.any && d < D ? p.b[col] : 0.f;
  }
  Source<T, false, VEC> o[K], z[K];
  auto load = [&](int64_t t) {
    const bool on = rw.any && t < p.T;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load_source<T, false, VEC, L>(o[k], p.o, t * p.o_st + rw.h * p.o_sh, nullptr, pl, k, D, on);
      if (p.z) load_source<T, false, VEC, L>(z[k], p.z, t * p.z_st + rw.h * p.z_sh, nullptr, pl, k, D, on);
    }
  };
  load(rw.t);
  for (; lead < p.T; lead += rw.step, rw.t += rw.step) {
    const bool on = rw.any && rw.t < p.T;
    float v[8 * K], g[8 * K];
#pragma unroll
    for (int i = 0; i < 8 * K; ++i) {
      v[i] = o[i / 8].get(i % 8);
      g[i] = p.z ? z[i / 8].get(i % 8) : 0.f;
    }
    load(rw.t + rw.step);
    float m = 0.f, s = 0.f;
    if (p.center) {
#pragma unroll
      for (int i = 0; i < 8 * K; ++i) s += v[i];
      m = group_sum<L>(s, red, turn) * p.inv_d;
    }
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * K; ++i) {
      const float x = v[i] - m;
      if (!p.center || pl.at(i / 8, i % 8) < D) s = fmaf(x, x, s);
    }
    const float r = rsqrtf(group_sum<L>(s, red, turn) * p.inv_d + p.eps);
    const int64_t row = rw.t * p.H + rw.h;
    if (p.o_codes) {
#pragma unroll
      for (int k = 0; k < K; ++k) save_eight<VEC, L>(v + 8 * k, p.o_codes + row * p.D, p.o_scales + row * blocks, pl, k, D, on);
      if (p.z) {
#pragma unroll
        for (int k = 0; k < K; ++k) save_eight<VEC, L>(g + 8 * k, p.z_codes + row * p.D, p.z_scales + row * blocks, pl, k, D, on);
      }
    }
#pragma unroll
    for (int i = 0; i < 8 * K; ++i) v[i] = fmaf((v[i] - m) * r, w[i], b[i]);
    if (p.z) {
      if (p.act == GDP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8 * K; ++i) v[i] *= g[i] * sigmoid(g[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8 * K; ++i) v[i] *= sigmoid(g[i]);
      }
    } else if (p.act == GDP_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < 8 * K; ++i) v[i] *= sigmoid(v[i]);
    }
    if (on) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Eight<T> e;
#pragma unroll
        for (int j = 0; j < 8; ++j) e.v[j] = from_f32<T>(v[8 * k + j]);
        store_eight<T, VEC, L>(static_cast<T *>(p.y) + row * p.D, e, pl, k, D);
      }
    }
  }
}

template <typename T, bool Q8, bool VEC, int L, int K>
__global__ void __launch_bounds__(kNormThreads<L>, K == 1 && L > 0 ? BWDB : 1) gdp_norm_bwd_kernel(const NormProblem p) {
  __shared__ float red[2][32];
  __shared__ float cols[L > 0 ? 2 * 8 * kNormThreads<L> : 1];
  int turn = 0;
  const Place<VEC, L> pl;
  const int D = (int)p.D;
  RowWalk rw(p, L > 0 ? (int)blockDim.x / (L > 0 ? L : 1) : 1, L);
  int64_t lead = L > 0 ? ((int64_t)blockIdx.x * blockDim.x + (threadIdx.x & ~31u)) / (L > 0 ? L : 1) / p.heads : rw.t;
  const int64_t blocks = (p.D + kBlock - 1) / kBlock;
  const bool zed = Q8 ? p.z_codes_in != nullptr : p.z != nullptr;
  float w[8 * K], b[8 * K], sw[8 * K], sb[8 * K];
#pragma unroll
  for (int i = 0; i < 8 * K; ++i) {
    const int d = pl.at(i / 8, i % 8);
    const int64_t col = (p.per_head ? rw.h * p.D : 0) + d;
    w[i] = rw.any && d < D ? p.w[col] : 0.f;
    b[i] = p.b && rw.any && d < D ? p.b[col] : 0.f;
    sw[i] = sb[i] = 0.f;
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
  for (; lead < p.T; lead += rw.step, rw.t += rw.step) {
    const bool on = rw.any && rw.t < p.T;
    float n[8 * K], g[8 * K], dn[8 * K];
#pragma unroll
    for (int i = 0; i < 8 * K; ++i) {
      n[i] = o[i / 8].get(i % 8);
      g[i] = zed ? z[i / 8].get(i % 8) : 0.f;
      dn[i] = to_f32(y[i / 8].v[i % 8]);
    }
    load(rw.t + rw.step);
    float m = 0.f, s = 0.f;
    if (p.center) {
#pragma unroll
      for (int i = 0; i < 8 * K; ++i) s += n[i];
      m = group_sum<L>(s, red, turn) * p.inv_d;
    }
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * K; ++i) {
      n[i] -= m;
      if (!p.center || pl.at(i / 8, i % 8) < D) s = fmaf(n[i], n[i], s);
    }
    const float r = rsqrtf(group_sum<L>(s, red, turn) * p.inv_d + p.eps);
    // dn: first dy, then du = dL/du, then du w; g: first z, then dz
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * K; ++i) {
      n[i] *= r;
      if (p.act != GDP_ACT_NONE) {
        const float u = fmaf(n[i], w[i], b[i]), x = zed ? g[i] : u;
        float q, rest;  // sigmoid(x) and 1 - sigmoid(x), each to its own relative precision
        gate_eval<GDP_GATE_SIGMOID>(x, &q, &rest);
        const float slope = p.act == GDP_ACT_SILU ? q * fmaf(x, rest, 1.f) : q * rest;
        if (zed) {
          g[i] = dn[i] * u * slope;
          dn[i] *= p.act == GDP_ACT_SILU ? x * q : q;
        } else {
          dn[i] *= slope;
        }
      }
      if (on) {
        sw[i] = fmaf(dn[i], n[i], sw[i]);
        if (p.b) sb[i] += dn[i];
      }
      dn[i] *= w[i];
      s1 += dn[i];
      s2 = fmaf(dn[i], n[i], s2);
    }
    s1 = p.center ? group_sum<L>(s1, red, turn) * p.inv_d : 0.f;
    s2 = group_sum<L>(s2, red, turn) * p.inv_d;
    if (on) {
      const int64_t row = rw.t * p.H + rw.h;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Eight<T> e;
#pragma unroll
        for (int j = 0; j < 8; ++j) e.v[j] = from_f32<T>(r * (dn[8 * k + j] - s1 - n[8 * k + j] * s2));
        store_eight<T, VEC, L>(static_cast<T *>(p.d_o) + row * p.D, e, pl, k, D);
        if (zed) {
#pragma unroll
          for (int j = 0; j < 8; ++j) e.v[j] = from_f32<T>(g[8 * k + j]);
          store_eight<T, VEC, L>(static_cast<T *>(p.d_z) + row * p.D, e, pl, k, D);
        }
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
        p.partial[part * ncols + off + d] = sw[i];
        if (p.b) p.partial[(p.parts + part) * ncols + off + d] = sb[i];
      }
    }
  } else if constexpr (L > 0) {  // one part per CTA: the groups' sums in turn
    constexpr int kGroups = kNormThreads<L> / L;
    const int group = (int)threadIdx.x / L;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cols[group * 8 * L + pl.at(0, j)] = rw.any ? sw[j] : 0.f;
      cols[(kGroups + group) * 8 * L + pl.at(0, j)] = rw.any ? sb[j] : 0.f;
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
