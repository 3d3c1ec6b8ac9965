// gdp_resnorm_body.cuh -- the residual norm's kernels, instantiated by type in gdp_resnorm_*.cu.
//
// A row belongs to a warp (up to 256 channels) or to a CTA (backward beyond 4096: to a pair of them); a thread holds eight
// of its channels in registers, so that every tensor is read once and the norms cost one reduction over the row each (backward
// too: the squares of both norms together, then the means of both).  Rows come ahead by asynchronous copies into places of
// shared memory that are the thread's own.  Bound by memory at last (36 bytes a channel of a training step with an fp32 stream,
// 14 forward and 22 backward), but first by instructions and the sums' latency: hence paired arithmetic, weights that stay in registers (forward) or shared memory (backward) instead of an L1 that the places leave
// too small, and two rows side by side in the forward pass, which share their sums' barriers.
//
// 65536 x 4096 bf16 with gate, scale and both weights, fp32 stream: forward 728 us, 5.2 TB/s (weights by way of L1, one row at a
// time: 858); backward 1300 us, 4.5 TB/s (weights by way of L1: 1763), bound by the latency of a row's two sums at 16 warps per SM.
// 32768 x 4096 with an fp32 stream: f16 rows 364 and 665 us, fp32 rows 628 (5.1 TB/s) and 1137 (4.2).  Rows of no 16-byte alignment
// go by elements: 1421 x 1601 f16 in 11.7 us, where its bytes take 4.0.
#pragma once

#include "gdp_resnorm.cuh"

namespace gdp {
namespace layer {

constexpr int kPairs = kRes / 2;

// Channel of a thread's value k: eight in a row where rows can be read by vectors, else `threads` apart.
template <bool VEC>
__device__ __forceinline__ int res_channel(int thread, int threads, int k) { return VEC ? thread * kRes + k : thread + k * threads; }

struct Eight {
  float2 v[kPairs];
};
__device__ __forceinline__ Eight eight_of(float v) {
  Eight e;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) e.v[k] = both(v);
  return e;
}
__device__ __forceinline__ float &value(Eight &e, int k) { return k % 2 ? e.v[k / 2].y : e.v[k / 2].x; }
__device__ __forceinline__ Eight operator*(const Eight &a, const Eight &b) {
  Eight e;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) e.v[k] = mul2(a.v[k], b.v[k]);
  return e;
}
__device__ __forceinline__ Eight operator*(const Eight &a, float b) {
  Eight e;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) e.v[k] = mul2(a.v[k], both(b));
  return e;
}
// a b + c
__device__ __forceinline__ Eight fma8(const Eight &a, const Eight &b, const Eight &c) {
  Eight e;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) e.v[k] = fma2(a.v[k], b.v[k], c.v[k]);
  return e;
}
__device__ __forceinline__ Eight add8(const Eight &a, const Eight &b) {
  Eight e;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) e.v[k] = add2(a.v[k], b.v[k]);
  return e;
}
__device__ __forceinline__ float dot(const Eight &a, const Eight &b) {
  float2 s = mul2(a.v[0], b.v[0]);
#pragma unroll
  for (int k = 1; k < kPairs; ++k) s = fma2(a.v[k], b.v[k], s);
  return s.x + s.y;
}

// ---- rows in global memory ----
// The thread's part of row t: one wide multiply, instead of pointers that would take registers (rows and strides are held
// below 2^31 by the host).
template <typename T, bool VEC>
__device__ __forceinline__ const T *row_at(const void *base, uint32_t t, int64_t stride, int thread = threadIdx.x) {
  return static_cast<const T *>(base) + (int64_t)(int)t * (int)stride + (VEC ? thread * kRes : 0);
}
template <typename T>
__device__ __forceinline__ T *out_at(void *base, uint32_t t, int C) { return static_cast<T *>(base) + (int64_t)(int)t * C; }

template <typename T, bool VEC>
__device__ __forceinline__ Eight load_row(const void *row, int thread, int threads, int C) {
  const T *at = static_cast<const T *>(row);
  Eight e = eight_of(0.f);
#pragma unroll
  for (int k = 0; k < kRes; ++k) {
    const int c = res_channel<VEC>(thread, threads, k);
    if (c < C) value(e, k) = to_f32(at[c]);
  }
  return e;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_row(void *row, int thread, int threads, int C, const Eight &e) {
  T *at = static_cast<T *>(row);
  if constexpr (VEC) {
    if (thread * kRes >= C) return;
    if constexpr (sizeof(T) == 4) {
      float4 *to = reinterpret_cast<float4 *>(at + thread * kRes);
      to[0] = make_float4(e.v[0].x, e.v[0].y, e.v[1].x, e.v[1].y);
      to[1] = make_float4(e.v[2].x, e.v[2].y, e.v[3].x, e.v[3].y);
    } else {
      *reinterpret_cast<uint4 *>(at + thread * kRes) = make_uint4(narrow<T>(e.v[0]), narrow<T>(e.v[1]), narrow<T>(e.v[2]), narrow<T>(e.v[3]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < kRes; ++k) {
      const int c = thread + k * threads;
      if (c < C) at[c] = from_f32<T>(k % 2 ? e.v[k / 2].y : e.v[k / 2].x);
    }
  }
}
// Columns of an fp32 vector; `other` where it is missing or has ended.
template <bool VEC>
__device__ __forceinline__ Eight load_columns(const float *at, int thread, int threads, int C, float other, int quad) {
  if (!at) return eight_of(other);
  Eight e = eight_of(other);
  if (VEC && quad) {
    if (thread * kRes < C) {
      const float4 a = reinterpret_cast<const float4 *>(at + thread * kRes)[0], b = reinterpret_cast<const float4 *>(at + thread * kRes)[1];
      e.v[0] = make_float2(a.x, a.y), e.v[1] = make_float2(a.z, a.w), e.v[2] = make_float2(b.x, b.y), e.v[3] = make_float2(b.z, b.w);
    }
    return e;
  }
#pragma unroll
  for (int k = 0; k < kRes; ++k) {
    const int c = res_channel<VEC>(thread, threads, k);
    if (c < C) value(e, k) = at[c];
  }
  return e;
}

// ---- rows on their way ----
// `depth` places per thread, three or two, so that depth - 1 rows are under way.  A place is some
// pieces of 16 bytes, a CTA's threads side by side in each.
struct RowPlaces {
  unsigned char *own;
  int piece, place, depth;  // bytes from one to the next
  __device__ __forceinline__ RowPlaces(unsigned char *smem, int pieces, int depth_) : depth(depth_) {
    own = smem + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
    piece = (int)(blockDim.x * blockDim.y) * 16;
    place = pieces * piece;
  }
  // a tensor's part of a row into pieces from `k` on
  template <int BYTES>
  __device__ __forceinline__ void ask(int p, int k, const void *from) const {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) sm100::cp_async16(own + p * place + (k + i) * piece, static_cast<const unsigned char *>(from) + 16 * i, 16u);
  }
  __device__ __forceinline__ void close() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
  __device__ __forceinline__ void wait() const {  // the oldest row of those under way has come
    if (depth == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  template <typename T>
  __device__ __forceinline__ Eight get(int p, int k) const {
    const unsigned char *at = own + p * place + k * piece;
    Eight e;
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4 *>(at), b = *reinterpret_cast<const float4 *>(at + piece);
      e.v[0] = make_float2(a.x, a.y), e.v[1] = make_float2(a.z, a.w), e.v[2] = make_float2(b.x, b.y), e.v[3] = make_float2(b.z, b.w);
    } else {
      const uint4 a = *reinterpret_cast<const uint4 *>(at);
      e.v[0] = widen<T>(a.x), e.v[1] = widen<T>(a.y), e.v[2] = widen<T>(a.z), e.v[3] = widen<T>(a.w);
    }
    return e;
  }
};

// ---- sums over a row ----
// Over its threads (WARPS 1: one warp), the same bits in all of them.  Two buffers in turn, so that one barrier per sum
// suffices; a buffer's places that no warp has stay zero.  A pair of CTAs (CL 2) writes its warps' sums into both buffers.
constexpr int kMostSums = 5;
template <int WARPS, int CL = 1>
struct RowSums {
  static constexpr int PLACES = WARPS < 4 ? 4 : WARPS;
  float (*buffer)[kMostSums][PLACES];
  int turn;
  uint32_t peer;  // CL 2: the other CTA's buffer, and the row's warps before this CTA's
  int before;
  __device__ __forceinline__ explicit RowSums(float (*b)[kMostSums][PLACES], int rank = 0) : buffer(b), turn(0), peer(0), before(rank * (WARPS / CL)) {
    if constexpr (WARPS > 1) {
      for (int i = threadIdx.x; i < 2 * kMostSums * PLACES; i += blockDim.x) (&buffer[0][0][0])[i] = 0.f;
      if constexpr (CL > 1) asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(sm100::smem_u32(buffer)), "r"(rank ^ 1));
      meet();
    }
  }
  __device__ __forceinline__ void meet() const {
    if constexpr (CL > 1) {
      __syncwarp();
      asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
  }
  // N sums, up to kMostSums.  Across warps: four warps' sums a lane, then over the lanes that hold the others.
  template <int N>
  __device__ __forceinline__ void over(float (&v)[N]) {
#pragma unroll
    for (int k = 16; k > 0; k /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], k);
    if constexpr (WARPS > 1) {
      if (threadIdx.x % 32 == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if constexpr (CL > 1) {
            buffer[turn][i][before + threadIdx.x / 32] = v[i];
            const uint32_t to = peer + ((turn * kMostSums + i) * PLACES + before + threadIdx.x / 32) * 4;
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v[i]) : "memory");
          } else {
            buffer[turn][i][threadIdx.x / 32] = v[i];
          }
        }
      meet();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float4 q = *reinterpret_cast<const float4 *>(&buffer[turn][i][threadIdx.x % (WARPS / 4) * 4]);
        v[i] = (q.x + q.y) + (q.z + q.w);
      }
#pragma unroll
      for (int k = 1; k < WARPS / 4; k *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], k);
      turn ^= 1;
    }
  }
};

// The gate's factor, and its slope.
__device__ __forceinline__ Eight gate_of(const Eight &g, int act) {
  if (act == GDP_ACT_NONE) return g;
  Eight e;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) e.v[k] = sigmoid2(g.v[k]);
  return act == GDP_ACT_SILU ? e * g : e;
}
__device__ __forceinline__ Eight gate_slope(const Eight &g, int act, Eight *factor) {
  *factor = g;
  if (act == GDP_ACT_NONE) return eight_of(1.f);
  Eight q, slope;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    float2 rest;  // 1 - q to its own precision: a sigmoid's slope is q rest, also where the gate is all but open
    sigmoid_halves(g.v[k], &q.v[k], &rest);
    slope.v[k] = mul2(q.v[k], act == GDP_ACT_SILU ? fma2(g.v[k], rest, both(1.f)) : rest);
  }
  *factor = act == GDP_ACT_SILU ? q * g : q;
  return slope;
}

// TR: the residual's type; RW: rows side by side.
template <typename T, typename TR, bool VEC, int MOST, int RW>
__global__ void __launch_bounds__(MOST) gdp_res_fwd_kernel(const ResProblem p) {
  constexpr int WARPS = MOST > 128 ? MOST / 32 : 1, B = kRes * (int)sizeof(T), R = kRes * (int)sizeof(TR);
  __shared__ __align__(16) float buffer[2][kMostSums][RowSums<WARPS>::PLACES];
  extern __shared__ __align__(16) unsigned char smem[];
  RowSums<WARPS> sums(buffer);
  const int thread = threadIdx.x, threads = blockDim.x, C = (int)p.C;
  const bool mine = thread * kRes < C;
  const int pieces = B / 16 * (p.gate ? 2 : 1) + R / 16;
  const RowPlaces places(smem, pieces * RW, p.depth);
  // (unsigned: the row behind the last ones may be past 2^31)
  const uint32_t first = blockIdx.x * blockDim.y + threadIdx.y, step = gridDim.x * blockDim.y, T_ = (uint32_t)p.T;
  auto ask = [&](uint32_t t, int place) {
#pragma unroll
    for (int i = 0; i < RW; ++i)
      if (mine && t + i * step < T_) {
        places.ask<B>(place, i * pieces, row_at<T, VEC>(p.block, t + i * step, p.block_st));
        places.ask<R>(place, i * pieces + B / 16, row_at<TR, VEC>(p.res, t + i * step, p.res_st));
        if (p.gate) places.ask<B>(place, i * pieces + B / 16 + R / 16, row_at<T, VEC>(p.gate, t + i * step, p.gate_st));
      }
    places.close();
  };
  if (VEC)
    for (int k = 0; k + 1 < p.depth; ++k) ask(first + k * RW * step, k);
  constexpr bool KEEP = RW > 1;  // weights in registers
  Eight post, scale, w;
  if (KEEP) {
    post = load_columns<VEC>(p.post, thread, threads, C, 0.f, p.quad_cols);
    scale = load_columns<VEC>(p.scale, thread, threads, C, 0.f, p.quad_cols);
    w = load_columns<VEC>(p.w, thread, threads, C, 0.f, p.quad_cols);
  }
  // MERGED: the block's sums are added up together with the stream's of the row before, so that a row has one barrier (CTAs of
  // more than 512 threads: 32768 x 8192 1044 to 812 us; where two rows share the barriers it costs: 65536 x 4096 733 to 754).
  constexpr bool MERGED = VEC && MOST > 512;
  auto squares = [&](uint32_t t, int at, float *s) {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      Eight m = eight_of(0.f);
      if (mine && t + i * step < T_) m = places.get<T>(at, i * pieces);
      s[i] = dot(m, m);
    }
  };
  float norm[RW];  // the block's sums
  const bool merged = MERGED && p.post;
  int place = 0;
  if (merged) {
    places.wait();
    squares(first, 0, norm);
    sums.over(norm);
  }
  for (uint32_t t = first; t < T_; t += RW * step) {
    Eight m[RW], r[RW], g[RW];
    const int after = place + 1 == p.depth ? 0 : place + 1;
#pragma unroll
    for (int i = 0; i < RW; ++i) m[i] = r[i] = g[i] = eight_of(0.f);
    if constexpr (VEC) {
      if (!merged) places.wait();
      ask(t + (p.depth - 1) * RW * step, place == 0 ? p.depth - 1 : place - 1);
#pragma unroll
      for (int i = 0; i < RW; ++i)
        if (mine && t + i * step < T_) {
          m[i] = places.get<T>(place, i * pieces);
          r[i] = places.get<TR>(place, i * pieces + B / 16);
          if (p.gate) g[i] = places.get<T>(place, i * pieces + B / 16 + R / 16);
        }
    } else {
      m[0] = load_row<T, VEC>(row_at<T, VEC>(p.block, t, p.block_st), thread, threads, C);
      r[0] = load_row<TR, VEC>(row_at<TR, VEC>(p.res, t, p.res_st), thread, threads, C);
      if (p.gate) g[0] = load_row<T, VEC>(row_at<T, VEC>(p.gate, t, p.gate_st), thread, threads, C);
    }
    float s[2 * RW];
    if (p.post) {
      if (!KEEP) post = load_columns<VEC>(p.post, thread, threads, C, 0.f, p.quad_cols);
      if (!merged) {
#pragma unroll
        for (int i = 0; i < RW; ++i) norm[i] = dot(m[i], m[i]);
        sums.over(norm);
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) m[i] = m[i] * post * rsqrtf(fmaf(norm[i], p.inv_c, p.eps));
    }
    if (p.gate)
#pragma unroll
      for (int i = 0; i < RW; ++i) m[i] = m[i] * gate_of(g[i], p.act);
    if (p.scale) {
      if (!KEEP) scale = load_columns<VEC>(p.scale, thread, threads, C, 0.f, p.quad_cols);
#pragma unroll
      for (int i = 0; i < RW; ++i) m[i] = m[i] * scale;
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      if (!VEC || mine) r[i] = add8(r[i], m[i]);
      s[i] = dot(r[i], r[i]);
      if (t + i * step < T_) store_row<TR, VEC>(out_at<TR>(p.r, t + i * step, C), thread, threads, C, r[i]);
    }
    if (!KEEP) w = load_columns<VEC>(p.w, thread, threads, C, 0.f, p.quad_cols);
    if (merged) {
      places.wait();
      squares(t + RW * step, after, s + RW);
      sums.over(s);
#pragma unroll
      for (int i = 0; i < RW; ++i) norm[i] = s[RW + i];
    } else {
      float only[RW];
#pragma unroll
      for (int i = 0; i < RW; ++i) only[i] = s[i];
      sums.over(only);
#pragma unroll
      for (int i = 0; i < RW; ++i) s[i] = only[i];
    }
#pragma unroll
    for (int i = 0; i < RW; ++i)
      if (t + i * step < T_)
        store_row<T, VEC>(out_at<T>(p.y, t + i * step, C), thread, threads, C, r[i] * w * rsqrtf(fmaf(s[i], p.inv_c, p.eps)));
    place = after;
  }
}

template <typename T, typename TR, bool VEC, int MOST, int CL>
__global__ void __launch_bounds__(MOST, MOST == 128 ? kResResident / MOST : 1) gdp_res_bwd_kernel(const ResProblem p) {
  constexpr int WARPS = MOST > 128 ? CL * MOST / 32 : 1, B = kRes * (int)sizeof(T), R = kRes * (int)sizeof(TR), PB = B / 16, PR = R / 16;
  __shared__ __align__(16) float buffer[2][kMostSums][RowSums<WARPS, CL>::PLACES];
  extern __shared__ __align__(16) unsigned char smem[];
  const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;  // (clusters are consecutive CTAs)
  RowSums<WARPS, CL> sums(buffer, rank);
  const int thread = rank * blockDim.x + threadIdx.x, threads = CL * blockDim.x, C = (int)p.C;
  const bool mine = thread * kRes < C;
  // pieces: dy, block, r, gate, dr
  const int dr_at = PB * (p.gate ? 3 : 2) + PR;
  const RowPlaces places(smem, dr_at + (p.dr ? PR : 0), p.depth);
  // weights of the thread's channels, behind the rows: two pieces each
  unsigned char *kept = smem + p.depth * places.place;
  const RowPlaces columns(kept, 6, 1);
  auto column = [&](int k) { return columns.get<float>(0, 2 * k); };
  if constexpr (VEC) {
    auto put = [&](int k, const Eight &e) {
      float4 *a = reinterpret_cast<float4 *>(columns.own + 2 * k * columns.piece), *b = reinterpret_cast<float4 *>(columns.own + (2 * k + 1) * columns.piece);
      *a = make_float4(e.v[0].x, e.v[0].y, e.v[1].x, e.v[1].y);
      *b = make_float4(e.v[2].x, e.v[2].y, e.v[3].x, e.v[3].y);
    };
    put(0, load_columns<VEC>(p.w, thread, threads, C, 0.f, p.quad_cols));
    put(1, load_columns<VEC>(p.post, thread, threads, C, 1.f, p.quad_cols));
    put(2, load_columns<VEC>(p.scale, thread, threads, C, 1.f, p.quad_cols));
  }
  auto weights = [&](int k, const float *from, float other) {
    return VEC ? column(k) : load_columns<VEC>(from, thread, threads, C, other, p.quad_cols);
  };
  // (unsigned: the row behind the last ones may be past 2^31)
  const uint32_t first = blockIdx.x / CL * blockDim.y + threadIdx.y, step = gridDim.x / CL * blockDim.y, T_ = (uint32_t)p.T;
  auto ask = [&](uint32_t t, int place) {
    if (mine && t < T_) {
      places.ask<B>(place, 0, row_at<T, VEC>(p.dy, t, p.dy_st, thread));
      places.ask<B>(place, PB, row_at<T, VEC>(p.block, t, p.block_st, thread));
      places.ask<R>(place, 2 * PB, row_at<TR, VEC>(p.res, t, p.res_st, thread));
      if (p.gate) places.ask<B>(place, 2 * PB + PR, row_at<T, VEC>(p.gate, t, p.gate_st, thread));
      if (p.dr) places.ask<R>(place, dr_at, row_at<TR, VEC>(p.dr, t, p.dr_st, thread));
    }
    places.close();
  };
  if (VEC)
    for (int k = 0; k + 1 < p.depth; ++k) ask(first + k * step, k);
  // MERGED: the norms' sums of a row are added up together with the means of the row before, so that a row has one barrier
  // (pairs of CTAs, whose barriers cost more: 32768 x 8192 2062 to 1554 us; one CTA, 65536 x 4096: 1327 to 1351).
  constexpr bool MERGED = VEC && CL > 1;
  auto squares = [&](int at, float *s) {
    Eight n = eight_of(0.f), m = n;
    if (mine) {
      m = places.get<T>(at, PB);
      n = places.get<TR>(at, 2 * PB);
    }
    s[0] = dot(n, n);
    s[1] = dot(m, m);
  };
  int place = 0;
  float s[2] = {0.f, 0.f};
  if constexpr (MERGED) {
    places.wait();
    if (first < T_) squares(0, s);
    sums.over(s);
  }
  Eight dw = eight_of(0.f), dpost = dw, dscale = dw;
  for (uint32_t t = first; t < T_; t += step) {
    Eight n = eight_of(0.f), m = n, d = n, g = n, up = n;
    const int after = place + 1 == p.depth ? 0 : place + 1;
    if constexpr (VEC) {
      if (!MERGED) places.wait();
      ask(t + (p.depth - 1) * step, place == 0 ? p.depth - 1 : place - 1);
      if (mine) {
        d = places.get<T>(place, 0);
        m = places.get<T>(place, PB);
        n = places.get<TR>(place, 2 * PB);
      }
    } else {
      d = load_row<T, VEC>(row_at<T, VEC>(p.dy, t, p.dy_st, thread), thread, threads, C);
      m = load_row<T, VEC>(row_at<T, VEC>(p.block, t, p.block_st, thread), thread, threads, C);
      n = load_row<TR, VEC>(row_at<TR, VEC>(p.res, t, p.res_st, thread), thread, threads, C);
      if (p.gate) g = load_row<T, VEC>(row_at<T, VEC>(p.gate, t, p.gate_st, thread), thread, threads, C);
      if (p.dr) up = load_row<TR, VEC>(row_at<TR, VEC>(p.dr, t, p.dr_st, thread), thread, threads, C);
    }
    // The second norm: n its normed values.  The stream's gradient is  d_r = r (d w - n mean(d w n)) + up, and what goes on
    // to the first norm's values m is d_r k with k = scale act(gate) post.  Its own mean(d_r k m) is linear in the other
    // mean, so that one pass over the row gives both:  mean((r d w + up) k m) - r mean(d w n) mean(n k m).
    const Eight w = weights(0, p.w, 0.f);
    if (!MERGED) {
      s[0] = dot(n, n);
      s[1] = dot(m, m);
    }
    if (VEC && mine) {
      if (p.gate) g = places.get<T>(place, 2 * PB + PR);
      if (p.dr) up = places.get<TR>(place, dr_at);
    }
    if (!MERGED) sums.over(s);
    const float r = rsqrtf(fmaf(s[0], p.inv_c, p.eps)), q = p.post ? rsqrtf(fmaf(s[1], p.inv_c, p.eps)) : 1.f;
    n = n * r;
    m = m * q;
    dw = fma8(d, n, dw);
    d = d * w;
    Eight a = eight_of(1.f), slope = a;
    if (p.gate) slope = gate_slope(g, p.act, &a);
    const Eight post = weights(1, p.post, 1.f), scale = weights(2, p.scale, 1.f);
    const Eight u = m * post;          // what gate and scale multiply
    up = fma8(d, eight_of(r), up);     // d_r but for its mean
    float means[MERGED ? kMostSums : 3] = {dot(d, n), 0.f, 0.f};
    if (p.post) {
      const Eight ku = a * scale * u;  // k m
      means[1] = dot(up, ku);
      means[2] = dot(n, ku);
    }
    if constexpr (MERGED) {
      places.wait();
      if (t + step < T_) squares(after, means + 3);
      sums.over(means);
      s[0] = means[3];
      s[1] = means[4];
    } else if (p.post) {
      sums.over(means);
    } else {
      float first_mean[1] = {means[0]};
      sums.over(first_mean);
      means[0] = first_mean[0];
    }
    place = after;
    const float back = -r * means[0] * p.inv_c;
    d = fma8(n, eight_of(back), up);
    store_row<TR, VEC>(out_at<TR>(p.dres, t, C), thread, threads, C, d);
    if (p.gate) store_row<T, VEC>(out_at<T>(p.dgate, t, C), thread, threads, C, d * scale * u * slope);
    d = d * a;
    if (p.scale) {
      dscale = fma8(d, u, dscale);
      d = d * scale;
    }
    if (p.post) {
      dpost = fma8(d, m, dpost);
      const float mean = fmaf(back, means[2], means[1]) * p.inv_c;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) d.v[k] = mul2(fma2(m.v[k], both(-mean), mul2(d.v[k], post.v[k])), both(q));
    }
    store_row<T, VEC>(out_at<T>(p.dblock, t, C), thread, threads, C, d);
  }
  if (CL > 1) sums.meet();  // the other CTA may still write here
  float *out = p.partial + (int64_t)(blockIdx.x / CL) * 3 * C;
  if constexpr (WARPS == 1) {  // the CTA's warps' sums, one after the other
    float *rows = reinterpret_cast<float *>(smem);
    if (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRes; ++k) {
      float *at = rows + threadIdx.y * 3 * 256 + k * 32 + thread;
      at[0] = value(dw, k);
      at[256] = value(dpost, k);
      at[512] = value(dscale, k);
    }
    __syncthreads();
    if (threadIdx.y != 0) return;
    for (int w = 1; w < blockDim.y; ++w)
#pragma unroll
      for (int k = 0; k < kRes; ++k) {
        const float *at = rows + w * 3 * 256 + k * 32 + thread;
        value(dw, k) += at[0];
        value(dpost, k) += at[256];
        value(dscale, k) += at[512];
      }
  }
#pragma unroll
  for (int k = 0; k < kRes; ++k) {
    const int c = res_channel<VEC>(thread, threads, k);
    if (c < C) {
      out[c] = value(dw, k);
      out[C + c] = value(dpost, k);
      out[2 * C + c] = value(dscale, k);
    }
  }
}

constexpr int kResShared = 226 * 1024;  // shared memory of an SM that CTAs' rows, weights and sums may take
constexpr int kResBeside = 2048;  // shared memory of a CTA besides its rows: the sums' buffers, and 1 KB of the system's
// Places of a row in shared memory (see RowPlaces) for `ctas` resident CTAs: three where there is room for them, or two, for
// which there is at every width, type and set of tensors.
inline int res_depth(int bytes, int ctas, int others) {
  const int room = kResShared / ctas - kResBeside - others;
  return 3 * bytes <= room ? 3 : 2;
}
// `rows`: CTAs or pairs of them.
template <int CL>
cudaError_t res_launch(void (*kernel)(ResProblem), const ResProblem &p, int64_t rows, dim3 block, int smem, cudaStream_t stream) {
  // (What is asked for and the kernel's own count together.  One limit for all calls: it is the kernel's, not the call's, and
  // another host thread may launch the same kernel with more.)
  if (smem + kResBeside > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kResShared - kResBeside);
    if (e != cudaSuccess) return e;
  }
  if constexpr (CL == 1) {
    kernel<<<(unsigned)rows, block, smem, stream>>>(p);
    return cudaGetLastError();
  } else {
    cudaLaunchConfig_t how{};
    how.gridDim = dim3((unsigned)(rows * CL));
    how.blockDim = block;
    how.dynamicSmemBytes = smem;
    how.stream = stream;
    cudaLaunchAttribute pair[1];
    pair[0].id = cudaLaunchAttributeClusterDimension;
    pair[0].val.clusterDim.x = CL;
    pair[0].val.clusterDim.y = pair[0].val.clusterDim.z = 1;
    how.attrs = pair;
    how.numAttrs = 1;
    return cudaLaunchKernelEx(&how, kernel, p);
  }
}
template <typename T, typename TR, int MOST>
cudaError_t res_fwd(ResProblem &p, int vec, cudaStream_t stream) {
  const dim3 block(res_threads(p.C, 1), res_rows(p.C));
  const int threads = block.x * block.y;
  const int row = threads * kRes * ((int)sizeof(T) * (p.gate ? 2 : 1) + (int)sizeof(TR));
  const int64_t rows = (p.T + block.y - 1) / block.y;
  if (!vec) return res_launch<1>(gdp_res_fwd_kernel<T, TR, false, MOST, 1>, p, rows, block, 0, stream);
  if constexpr (MOST == 512) {  // two rows side by side, where every SM has several pairs of them
    const int per_sm = 512 / threads > 1 ? 512 / threads : 1;
    const int64_t resident = (int64_t)sm_count() * per_sm;
    if (rows >= 8 * resident) {
      p.depth = res_depth(2 * row, per_sm, 0);
      return res_launch<1>(gdp_res_fwd_kernel<T, TR, true, MOST, 2>, p, resident, block, p.depth * 2 * row, stream);
    }
  }
  const int per_sm = 1024 / threads;
  p.depth = res_depth(row, per_sm, 0);
  const int64_t resident = (int64_t)sm_count() * per_sm;
  return res_launch<1>(gdp_res_fwd_kernel<T, TR, true, MOST, 1>, p, rows < resident ? rows : resident, block, p.depth * row, stream);
}
template <typename T, typename TR>
cudaError_t res_fwd_by(ResProblem &p, int vec, cudaStream_t stream) {
  if (res_rows(p.C) > 1) return res_fwd<T, TR, 128>(p, vec, stream);
  return res_threads(p.C, 1) <= 512 ? res_fwd<T, TR, 512>(p, vec, stream) : res_fwd<T, TR, 1024>(p, vec, stream);
}
template <typename T>
cudaError_t launch_res_fwd(ResProblem &p, int vec, cudaStream_t stream) {
  return p.res_f32 ? res_fwd_by<T, float>(p, vec, stream) : res_fwd_by<T, T>(p, vec, stream);
}
template <typename T, typename TR, int MOST, int CL>
cudaError_t res_bwd(ResProblem &p, int vec, int64_t parts, cudaStream_t stream) {
  const dim3 block(res_threads(p.C, CL), res_rows(p.C));
  const int threads = block.x * block.y, per_sm = kResResident / threads > 1 ? kResResident / threads : 1;
  const int row = threads * kRes * ((int)sizeof(T) * (p.gate ? 3 : 2) + (int)sizeof(TR) * (p.dr ? 2 : 1)), kept = threads * kRes * 3 * 4;
  p.depth = res_depth(row, per_sm, kept);
  const int sums = block.y > 1 ? (int)block.y * 3 * 256 * (int)sizeof(float) : 0;
  int smem = vec ? p.depth * row + kept : 0;
  if (smem < sums) smem = sums;
  return res_launch<CL>(vec ? gdp_res_bwd_kernel<T, TR, true, MOST, CL> : gdp_res_bwd_kernel<T, TR, false, MOST, CL>, p, parts, block, smem, stream);
}
template <typename T, typename TR>
cudaError_t res_bwd_by(ResProblem &p, int vec, int64_t parts, cudaStream_t stream) {
  if (res_rows(p.C) > 1) return res_bwd<T, TR, 128, 1>(p, vec, parts, stream);
  return res_cluster(p.C) == 1 ? res_bwd<T, TR, 512, 1>(p, vec, parts, stream) : res_bwd<T, TR, 512, 2>(p, vec, parts, stream);
}
template <typename T>
cudaError_t launch_res_bwd(ResProblem &p, int vec, int64_t parts, cudaStream_t stream) {
  return p.res_f32 ? res_bwd_by<T, float>(p, vec, parts, stream) : res_bwd_by<T, T>(p, vec, parts, stream);
}

}  // namespace layer
}  // namespace gdp
