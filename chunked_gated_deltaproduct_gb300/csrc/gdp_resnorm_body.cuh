// gdp_resnorm_body.cuh -- the residual norm's kernels, instantiated by type in gdp_resnorm_*.cu.
//
// A row belongs to a warp (up to 256 channels) or to a CTA; a thread holds eight of its channels in registers, so that
// every tensor is read once and the norms cost one reduction each (backward: three for the two).  Rows come ahead by
// asynchronous copies into places of shared memory that are the thread's own.  Bound by memory in the end, and on the way
// there by instructions: at 57 bytes a channel pair the SM has four issue slots for ... see the figures at the launchers.
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
// `depth` places per thread, so that depth - 1 rows are under way (depth 1: the row itself, waited for).  A place is some
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
// Over its threads (ONE: one warp), the same bits in all of them.  Two buffers in turn, so that one barrier per sum
// suffices; a buffer's places that no warp has stay zero.
template <int WARPS>
struct RowSums {
  static constexpr int PAIRS = (WARPS + 1) / 2 * 2;
  float2 (*buffer)[PAIRS];
  int turn;
  __device__ __forceinline__ explicit RowSums(float2 (*b)[PAIRS]) : buffer(b), turn(0) {
    if constexpr (WARPS > 1) {
      for (int i = threadIdx.x; i < 2 * PAIRS; i += blockDim.x) buffer[i / PAIRS][i % PAIRS] = make_float2(0.f, 0.f);
      __syncthreads();
    }
  }
  __device__ __forceinline__ float one(float v) {
#pragma unroll
    for (int k = 16; k > 0; k /= 2) v += __shfl_xor_sync(0xffffffffu, v, k);
    if constexpr (WARPS > 1) v = across(make_float2(v, 0.f)).x;
    return v;
  }
  __device__ __forceinline__ float2 two(float2 v) {
#pragma unroll
    for (int k = 16; k > 0; k /= 2) v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, k), __shfl_xor_sync(0xffffffffu, v.y, k)));
    if constexpr (WARPS > 1) v = across(v);
    return v;
  }
  __device__ __forceinline__ float2 across(float2 v) {
    if (threadIdx.x % 32 == 0) buffer[turn][threadIdx.x / 32] = v;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < PAIRS; k += 2) {
      const float4 q = *reinterpret_cast<const float4 *>(&buffer[turn][k]);
      s = add2(s, add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
    }
    turn ^= 1;
    return s;
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
    q.v[k] = sigmoid2(g.v[k]);
    const float2 rest = fma2(q.v[k], both(-1.f), both(1.f));
    slope.v[k] = mul2(q.v[k], act == GDP_ACT_SILU ? fma2(g.v[k], rest, both(1.f)) : rest);
  }
  *factor = act == GDP_ACT_SILU ? q * g : q;
  return slope;
}

// TR: the residual's type.
template <typename T, typename TR, bool VEC, int MOST>
__global__ void __launch_bounds__(MOST) gdp_res_fwd_kernel(const ResProblem p) {
  constexpr int WARPS = MOST > 128 ? MOST / 32 : 1, B = kRes * (int)sizeof(T), R = kRes * (int)sizeof(TR);
  __shared__ __align__(16) float2 buffer[2][RowSums<WARPS>::PAIRS];
  extern __shared__ __align__(16) unsigned char smem[];
  RowSums<WARPS> sums(buffer);
  const int thread = threadIdx.x, threads = blockDim.x, C = (int)p.C;
  const bool mine = thread * kRes < C;
  const RowPlaces places(smem, B / 16 * (p.gate ? 2 : 1) + R / 16, p.depth);
  const int64_t first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, step = (int64_t)gridDim.x * blockDim.y;
  const T *block = static_cast<const T *>(p.block) + first * p.block_st + (VEC ? thread * kRes : 0),
          *gate = static_cast<const T *>(p.gate) + (p.gate ? first * p.gate_st + (VEC ? thread * kRes : 0) : 0);
  const TR *res = static_cast<const TR *>(p.res) + first * p.res_st + (VEC ? thread * kRes : 0);
  T *y_to = static_cast<T *>(p.y) + first * p.C;
  TR *r_to = static_cast<TR *>(p.r) + first * p.C;
  int64_t asked = first;
  auto ask = [&](int place) {
    if (mine && asked < p.T) {
      places.ask<B>(place, 0, block);
      places.ask<R>(place, B / 16, res);
      if (p.gate) places.ask<B>(place, B / 16 + R / 16, gate);
    }
    asked += step;
    block += step * p.block_st;
    res += step * p.res_st;
    if (p.gate) gate += step * p.gate_st;
    places.close();
  };
  if (VEC)
    for (int k = 0; k + 1 < p.depth; ++k) ask(k);
  int place = 0;
  for (int64_t t = first; t < p.T; t += step, place = place + 1 == p.depth ? 0 : place + 1) {
    Eight m = eight_of(0.f), r = m, g = m;
    if constexpr (VEC) {
      if (p.depth == 1) ask(0);
      places.wait();
      if (p.depth > 1) ask(place == 0 ? p.depth - 1 : place - 1);
      if (mine) {
        m = places.get<T>(place, 0);
        r = places.get<TR>(place, B / 16);
        if (p.gate) g = places.get<T>(place, B / 16 + R / 16);
      }
    } else {
      m = load_row<T, VEC>(block, thread, threads, C);
      r = load_row<TR, VEC>(res, thread, threads, C);
      if (p.gate) g = load_row<T, VEC>(gate, thread, threads, C);
      block += step * p.block_st;
      res += step * p.res_st;
      if (p.gate) gate += step * p.gate_st;
    }
    if (p.post) {
      const Eight post = load_columns<VEC>(p.post, thread, threads, C, 0.f, p.quad_cols);
      m = m * post * rsqrtf(fmaf(sums.one(dot(m, m)), p.inv_c, p.eps));
    }
    if (p.gate) m = m * gate_of(g, p.act);
    if (p.scale) m = m * load_columns<VEC>(p.scale, thread, threads, C, 0.f, p.quad_cols);
    if (VEC ? mine : true) r = add8(r, m);
    store_row<TR, VEC>(r_to, thread, threads, C, r);
    const Eight w = load_columns<VEC>(p.w, thread, threads, C, 0.f, p.quad_cols);
    const float q = rsqrtf(fmaf(sums.one(dot(r, r)), p.inv_c, p.eps));
    store_row<T, VEC>(y_to, thread, threads, C, r * w * q);
    r_to += step * p.C;
    y_to += step * p.C;
  }
}

template <typename T, typename TR, bool VEC, int MOST>
__global__ void __launch_bounds__(MOST) gdp_res_bwd_kernel(const ResProblem p) {
  constexpr int WARPS = MOST > 128 ? MOST / 32 : 1, B = kRes * (int)sizeof(T), R = kRes * (int)sizeof(TR), PB = B / 16, PR = R / 16;
  __shared__ __align__(16) float2 buffer[2][RowSums<WARPS>::PAIRS];
  extern __shared__ __align__(16) unsigned char smem[];
  RowSums<WARPS> sums(buffer);
  const int thread = threadIdx.x, threads = blockDim.x, C = (int)p.C, lane = VEC ? thread * kRes : 0;
  const bool mine = thread * kRes < C;
  // pieces: dy, block, r, gate, dr
  const int dr_at = PB * (p.gate ? 3 : 2) + PR;
  const RowPlaces places(smem, dr_at + (p.dr ? PR : 0), p.depth);
  const int64_t first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, step = (int64_t)gridDim.x * blockDim.y;
  const T *dy = static_cast<const T *>(p.dy) + first * p.dy_st + lane, *block = static_cast<const T *>(p.block) + first * p.block_st + lane,
          *gate = static_cast<const T *>(p.gate) + (p.gate ? first * p.gate_st + lane : 0);
  const TR *res = static_cast<const TR *>(p.res) + first * p.res_st + lane, *dr = static_cast<const TR *>(p.dr) + (p.dr ? first * p.dr_st + lane : 0);
  TR *dres = static_cast<TR *>(p.dres) + first * p.C;
  T *dblock = static_cast<T *>(p.dblock) + first * p.C, *dgate = static_cast<T *>(p.dgate) + (p.gate ? first * p.C : 0);
  int64_t asked = first;
  auto advance = [&] {
    dy += step * p.dy_st;
    block += step * p.block_st;
    res += step * p.res_st;
    if (p.gate) gate += step * p.gate_st;
    if (p.dr) dr += step * p.dr_st;
  };
  auto ask = [&](int place) {
    if (mine && asked < p.T) {
      places.ask<B>(place, 0, dy);
      places.ask<B>(place, PB, block);
      places.ask<R>(place, 2 * PB, res);
      if (p.gate) places.ask<B>(place, 2 * PB + PR, gate);
      if (p.dr) places.ask<R>(place, dr_at, dr);
    }
    asked += step;
    advance();
    places.close();
  };
  if (VEC)
    for (int k = 0; k + 1 < p.depth; ++k) ask(k);
  int place = 0;
  Eight dw = eight_of(0.f), dpost = dw, dscale = dw;
  for (int64_t t = first; t < p.T; t += step, place = place + 1 == p.depth ? 0 : place + 1) {
    Eight n = eight_of(0.f), m = n, d = n, g = n, up = n;
    if constexpr (VEC) {
      if (p.depth == 1) ask(0);
      places.wait();
      if (p.depth > 1) ask(place == 0 ? p.depth - 1 : place - 1);
      if (mine) {
        d = places.get<T>(place, 0);
        m = places.get<T>(place, PB);
        n = places.get<TR>(place, 2 * PB);
      }
    } else {
      d = load_row<T, VEC>(dy, thread, threads, C);
      m = load_row<T, VEC>(block, thread, threads, C);
      n = load_row<TR, VEC>(res, thread, threads, C);
      if (p.gate) g = load_row<T, VEC>(gate, thread, threads, C);
      if (p.dr) up = load_row<TR, VEC>(dr, thread, threads, C);
      advance();
    }
    // the second norm: n becomes its normed values, d the gradient of the stream
    const Eight w = load_columns<VEC>(p.w, thread, threads, C, 0.f, p.quad_cols);
    const float2 s = sums.two(make_float2(dot(n, n), dot(m, m)));
    const float r = rsqrtf(fmaf(s.x, p.inv_c, p.eps)), q = p.post ? rsqrtf(fmaf(s.y, p.inv_c, p.eps)) : 1.f;
    n = n * r;
    dw = fma8(d, n, dw);
    d = d * w;
    if (VEC && mine && p.dr) up = places.get<TR>(place, dr_at);
    const Eight post = load_columns<VEC>(p.post, thread, threads, C, 1.f, p.quad_cols);
    float mean = sums.one(dot(d, n)) * p.inv_c;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) d.v[k] = fma2(fma2(n.v[k], both(-mean), d.v[k]), both(r), up.v[k]);
    store_row<TR, VEC>(dres, thread, threads, C, d);
    // the first one, under gate and scale: m its normed values, d becomes their gradient
    m = m * q;
    if (p.gate) {
      if (VEC && mine) g = places.get<T>(place, 2 * PB + PR);
      Eight a;
      const Eight slope = gate_slope(g, p.act, &a), u = m * post;
      Eight through = d;  // of the gated norm
      if (p.scale) through = d * load_columns<VEC>(p.scale, thread, threads, C, 1.f, p.quad_cols);
      store_row<T, VEC>(dgate, thread, threads, C, through * u * slope);
      if (p.scale) dscale = fma8(d * a, u, dscale);
      d = through * a;
      dgate += step * p.C;
    } else if (p.scale) {
      dscale = fma8(d, m * post, dscale);
      d = d * load_columns<VEC>(p.scale, thread, threads, C, 1.f, p.quad_cols);
    }
    if (p.post) {
      dpost = fma8(d, m, dpost);
      d = d * post;
      mean = sums.one(dot(d, m)) * p.inv_c;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) d.v[k] = mul2(fma2(m.v[k], both(-mean), d.v[k]), both(q));
    }
    store_row<T, VEC>(dblock, thread, threads, C, d);
    dres += step * p.C;
    dblock += step * p.C;
  }
  float *out = p.partial + (int64_t)blockIdx.x * 3 * C;
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

// Places of a row in shared memory (see RowPlaces) for `ctas` resident CTAs: three, or as many as there is room for.
inline int res_depth(int bytes, int ctas) {
  const int room = 226 * 1024 / ctas - 1024;
  return 3 * bytes <= room ? 3 : 2 * bytes <= room ? 2 : 1;
}
template <typename T, typename TR, int MOST>
cudaError_t res_fwd(ResProblem &p, int vec, cudaStream_t stream) {
  const dim3 block(res_threads(p.C), res_rows(p.C));
  const int threads = block.x * block.y, per_sm = 1024 / threads;
  const int row = threads * kRes * ((int)sizeof(T) * (p.gate ? 2 : 1) + (int)sizeof(TR));
  p.depth = res_depth(row, per_sm);
  const int smem = vec ? p.depth * row : 0;
  const int64_t rows = (p.T + block.y - 1) / block.y, resident = (int64_t)sm_count() * per_sm;
  const dim3 grid((unsigned)(rows < resident || !vec ? rows : resident));
  const auto kernel = vec ? gdp_res_fwd_kernel<T, TR, true, MOST> : gdp_res_fwd_kernel<T, TR, false, MOST>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, block, smem, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, typename TR>
cudaError_t res_fwd_by(ResProblem &p, int vec, cudaStream_t stream) {
  if (res_rows(p.C) > 1) return res_fwd<T, TR, 128>(p, vec, stream);
  return res_threads(p.C) <= 512 ? res_fwd<T, TR, 512>(p, vec, stream) : res_fwd<T, TR, 1024>(p, vec, stream);
}
template <typename T>
cudaError_t launch_res_fwd(ResProblem &p, int vec, cudaStream_t stream) {
  return p.res_f32 ? res_fwd_by<T, float>(p, vec, stream) : res_fwd_by<T, T>(p, vec, stream);
}
template <typename T, typename TR, int MOST>
cudaError_t res_bwd(ResProblem &p, int vec, int64_t ctas, cudaStream_t stream) {
  const dim3 block(res_threads(p.C), res_rows(p.C));
  const int threads = block.x * block.y;
  const int row = threads * kRes * ((int)sizeof(T) * (p.gate ? 3 : 2) + (int)sizeof(TR) * (p.dr ? 2 : 1));
  p.depth = res_depth(row, kResResident / threads > 1 ? kResResident / threads : 1);
  const int sums = block.y > 1 ? (int)block.y * 3 * 256 * (int)sizeof(float) : 0;
  int smem = vec ? p.depth * row : 0;
  if (smem < sums) smem = sums;
  const auto kernel = vec ? gdp_res_bwd_kernel<T, TR, true, MOST> : gdp_res_bwd_kernel<T, TR, false, MOST>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)ctas, block, smem, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, typename TR>
cudaError_t res_bwd_by(ResProblem &p, int vec, int64_t ctas, cudaStream_t stream) {
  if (res_rows(p.C) > 1) return res_bwd<T, TR, 128>(p, vec, ctas, stream);
  return res_threads(p.C) <= 512 ? res_bwd<T, TR, 512>(p, vec, ctas, stream) : res_bwd<T, TR, 1024>(p, vec, ctas, stream);
}
template <typename T>
cudaError_t launch_res_bwd(ResProblem &p, int vec, int64_t ctas, cudaStream_t stream) {
  return p.res_f32 ? res_bwd_by<T, float>(p, vec, ctas, stream) : res_bwd_by<T, T>(p, vec, ctas, stream);
}

}  // namespace layer
}  // namespace gdp
