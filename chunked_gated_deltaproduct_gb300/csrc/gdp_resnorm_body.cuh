// gdp_resnorm_body.cuh -- the residual norm's kernels, instantiated by type in gdp_resnorm_*.cu.
//
// A row belongs to a warp (up to 256 channels) or to a CTA; a thread holds eight of its channels in registers, so that
// every tensor is read once and the two norms cost two reductions of one value.
#pragma once

#include "gdp_resnorm.cuh"

namespace gdp {
namespace layer {

// Channel of a thread's value k: eight in a row where rows can be read by vectors, else `threads` apart.
template <bool VEC>
__device__ __forceinline__ int res_channel(int thread, int threads, int k) { return VEC ? thread * kRes + k : thread + k * threads; }

template <typename T, bool VEC>
__device__ __forceinline__ void load_row(const void *base, int64_t offset, int thread, int threads, int C, float (&v)[kRes]) {
  const T *at = static_cast<const T *>(base) + offset;
  if constexpr (VEC) {
    if (thread * kRes < C) {
      constexpr int Q = 16 / sizeof(T);
#pragma unroll
      for (int k = 0; k < kRes; k += Q) {
        const Vec<T, Q> q = load_vec<T, Q>(at + thread * kRes + k);
#pragma unroll
        for (int i = 0; i < Q; ++i) v[k + i] = to_f32(q.v[i]);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < kRes; ++k) v[k] = 0.f;
  } else {
#pragma unroll
    for (int k = 0; k < kRes; ++k) {
      const int c = thread + k * threads;
      v[k] = c < C ? to_f32(at[c]) : 0.f;
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_row(void *base, int64_t offset, int thread, int threads, int C, const float (&v)[kRes]) {
  T *at = static_cast<T *>(base) + offset;
  if constexpr (VEC) {
    if (thread * kRes < C) {
      constexpr int Q = 16 / sizeof(T);
#pragma unroll
      for (int k = 0; k < kRes; k += Q) store_vec<T, Q>(at + thread * kRes + k, v + k);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kRes; ++k) {
      const int c = thread + k * threads;
      if (c < C) at[c] = from_f32<T>(v[k]);
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_stream(const ResProblem &p, const void *base, int64_t offset, int thread, int threads, float (&v)[kRes]) {
  if (p.res_f32) load_row<float, VEC>(base, offset, thread, threads, (int)p.C, v);
  else load_row<T, VEC>(base, offset, thread, threads, (int)p.C, v);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_stream(const ResProblem &p, void *base, int64_t offset, int thread, int threads, const float (&v)[kRes]) {
  if (p.res_f32) store_row<float, VEC>(base, offset, thread, threads, (int)p.C, v);
  else store_row<T, VEC>(base, offset, thread, threads, (int)p.C, v);
}

// Sum over a row's threads (ONE: one warp), the same bits in all of them.  `spare` alternates between two buffers, so
// that one barrier per sum suffices.
template <bool ONE>
__device__ __forceinline__ float2 row_sum(float2 v, float2 (*buffer)[32], int &spare) {
#pragma unroll
  for (int k = 16; k > 0; k /= 2) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, k);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, k);
  }
  if constexpr (!ONE) {
    const int warps = blockDim.x / 32;
    if (threadIdx.x % 32 == 0) buffer[spare][threadIdx.x / 32] = v;
    __syncthreads();
    v = threadIdx.x % 32 < warps ? buffer[spare][threadIdx.x % 32] : make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 16; k > 0; k /= 2) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, k);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, k);
    }
    spare ^= 1;
  }
  return v;
}

template <bool VEC>
__device__ __forceinline__ void load_columns(const float *at, int thread, int threads, int C, float other, float (&v)[kRes]) {
#pragma unroll
  for (int k = 0; k < kRes; ++k) {
    const int c = res_channel<VEC>(thread, threads, k);
    v[k] = at && c < C ? at[c] : other;
  }
}

__device__ __forceinline__ float gate_of(float g, int act) {
  return act == GDP_ACT_NONE ? g : sigmoid_fast(g) * (act == GDP_ACT_SILU ? g : 1.f);
}
__device__ __forceinline__ float gate_slope(float g, int act) {
  if (act == GDP_ACT_NONE) return 1.f;
  const float q = sigmoid_fast(g);
  return act == GDP_ACT_SILU ? q * fmaf(g, 1.f - q, 1.f) : q * (1.f - q);
}

template <typename T, bool VEC, bool ONE, int MOST>
__global__ void __launch_bounds__(MOST) gdp_res_fwd_kernel(const ResProblem p) {
  __shared__ float2 buffer[2][32];
  int spare = 0;
  const int thread = threadIdx.x, threads = blockDim.x, C = (int)p.C;
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (ONE && t >= p.T) return;
  float m[kRes], r[kRes], col[kRes];
  load_row<T, VEC>(p.block, t * p.block_st, thread, threads, C, m);
  load_stream<T, VEC>(p, p.res, t * p.res_st, thread, threads, r);
  if (p.post) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kRes; ++k) s = fmaf(m[k], m[k], s);
    const float q = rsqrtf(row_sum<ONE>(make_float2(s, 0.f), buffer, spare).x * p.inv_c + p.eps);
    load_columns<VEC>(p.post, thread, threads, C, 0.f, col);
#pragma unroll
    for (int k = 0; k < kRes; ++k) m[k] *= q * col[k];
  }
  if (p.gate) {
    float g[kRes];
    load_row<T, VEC>(p.gate, t * p.gate_st, thread, threads, C, g);
#pragma unroll
    for (int k = 0; k < kRes; ++k) m[k] *= gate_of(g[k], p.act);
  }
  if (p.scale) {
    load_columns<VEC>(p.scale, thread, threads, C, 0.f, col);
#pragma unroll
    for (int k = 0; k < kRes; ++k) m[k] *= col[k];
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kRes; ++k) {
    r[k] += res_channel<VEC>(thread, threads, k) < C ? m[k] : 0.f;
    s = fmaf(r[k], r[k], s);
  }
  store_stream<T, VEC>(p, p.r, t * p.C, thread, threads, r);
  const float q = rsqrtf(row_sum<ONE>(make_float2(s, 0.f), buffer, spare).x * p.inv_c + p.eps);
  load_columns<VEC>(p.w, thread, threads, C, 0.f, col);
#pragma unroll
  for (int k = 0; k < kRes; ++k) r[k] *= q * col[k];
  store_row<T, VEC>(p.y, t * p.C, thread, threads, C, r);
}

template <typename T, bool VEC, bool ONE, int MOST>
__global__ void __launch_bounds__(MOST) gdp_res_bwd_kernel(const ResProblem p) {
  __shared__ float2 buffer[2][32];
  extern __shared__ float rows[];  // ONE: the column sums of the CTA's warps
  int spare = 0;
  const int thread = threadIdx.x, threads = blockDim.x, C = (int)p.C;
  float dw[kRes] = {}, dpost[kRes] = {}, dscale[kRes] = {};
  for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < p.T; t += (int64_t)gridDim.x * blockDim.y) {
    float n[kRes], m[kRes], d[kRes], col[kRes];
    load_stream<T, VEC>(p, p.res, t * p.res_st, thread, threads, n);
    load_row<T, VEC>(p.dy, t * p.dy_st, thread, threads, C, d);
    load_row<T, VEC>(p.block, t * p.block_st, thread, threads, C, m);
    // the second norm: n its normed values, r its reciprocal root
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kRes; ++k) {
      s.x = fmaf(n[k], n[k], s.x);
      s.y = fmaf(m[k], m[k], s.y);
    }
    s = row_sum<ONE>(s, buffer, spare);
    const float r = rsqrtf(s.x * p.inv_c + p.eps), q = p.post ? rsqrtf(s.y * p.inv_c + p.eps) : 1.f;
    load_columns<VEC>(p.w, thread, threads, C, 0.f, col);
    float mean = 0.f;
#pragma unroll
    for (int k = 0; k < kRes; ++k) {
      n[k] *= r;
      dw[k] = fmaf(d[k], n[k], dw[k]);
      d[k] *= col[k];
      mean = fmaf(d[k], n[k], mean);
    }
    mean = row_sum<ONE>(make_float2(mean, 0.f), buffer, spare).x * p.inv_c;
    float up[kRes] = {};
    if (p.dr) load_stream<T, VEC>(p, p.dr, t * p.dr_st, thread, threads, up);
#pragma unroll
    for (int k = 0; k < kRes; ++k) d[k] = fmaf(r, d[k] - n[k] * mean, up[k]);
    store_stream<T, VEC>(p, p.dres, t * p.C, thread, threads, d);
    // what it is multiplied with: d the gradient of the scaled and gated first norm, m its normed values
    float post[kRes], scale[kRes];
    load_columns<VEC>(p.post, thread, threads, C, 1.f, post);
    load_columns<VEC>(p.scale, thread, threads, C, 1.f, scale);
#pragma unroll
    for (int k = 0; k < kRes; ++k) m[k] *= q;
    if (p.gate) {
      float g[kRes], dg[kRes];
      load_row<T, VEC>(p.gate, t * p.gate_st, thread, threads, C, g);
#pragma unroll
      for (int k = 0; k < kRes; ++k) {
        const float a = gate_of(g[k], p.act), u = m[k] * post[k];
        dg[k] = d[k] * scale[k] * u * gate_slope(g[k], p.act);
        dscale[k] = fmaf(d[k] * a, u, dscale[k]);
        d[k] *= a * scale[k];
      }
      store_row<T, VEC>(p.dgate, t * p.C, thread, threads, C, dg);
    } else {
#pragma unroll
      for (int k = 0; k < kRes; ++k) {
        dscale[k] = fmaf(d[k], m[k] * post[k], dscale[k]);
        d[k] *= scale[k];
      }
    }
    if (p.post) {
      mean = 0.f;
#pragma unroll
      for (int k = 0; k < kRes; ++k) {
        dpost[k] = fmaf(d[k], m[k], dpost[k]);
        d[k] *= post[k];
        mean = fmaf(d[k], m[k], mean);
      }
      mean = row_sum<ONE>(make_float2(mean, 0.f), buffer, spare).x * p.inv_c;
#pragma unroll
      for (int k = 0; k < kRes; ++k) d[k] = q * (d[k] - m[k] * mean);
    }
    store_row<T, VEC>(p.dblock, t * p.C, thread, threads, C, d);
  }
  float *out = p.partial + (int64_t)blockIdx.x * 3 * C;
  if constexpr (ONE) {
#pragma unroll
    for (int k = 0; k < kRes; ++k) {
      float *at = rows + threadIdx.y * 3 * 256 + k * 32 + thread;
      at[0] = dw[k];
      at[256] = dpost[k];
      at[512] = dscale[k];
    }
    __syncthreads();
    if (threadIdx.y != 0) return;
    for (int w = 1; w < blockDim.y; ++w)
#pragma unroll
      for (int k = 0; k < kRes; ++k) {
        const float *at = rows + w * 3 * 256 + k * 32 + thread;
        dw[k] += at[0];
        dpost[k] += at[256];
        dscale[k] += at[512];
      }
  }
#pragma unroll
  for (int k = 0; k < kRes; ++k) {
    const int c = res_channel<VEC>(thread, threads, k);
    if (c < C) {
      out[c] = dw[k];
      out[C + c] = dpost[k];
      out[2 * C + c] = dscale[k];
    }
  }
}

template <typename T, bool ONE, int MOST>
void res_fwd(const ResProblem &p, int vec, dim3 grid, dim3 block, cudaStream_t stream) {
  if (vec) gdp_res_fwd_kernel<T, true, ONE, MOST><<<grid, block, 0, stream>>>(p);
  else gdp_res_fwd_kernel<T, false, ONE, MOST><<<grid, block, 0, stream>>>(p);
}
template <typename T>
cudaError_t launch_res_fwd(const ResProblem &p, int vec, cudaStream_t stream) {
  const dim3 block(res_threads(p.C), res_rows(p.C)), grid((unsigned)((p.T + block.y - 1) / block.y));
  if (block.y > 1) res_fwd<T, true, 128>(p, vec, grid, block, stream);
  else res_fwd<T, false, 1024>(p, vec, grid, block, stream);
  return cudaGetLastError();
}
template <typename T, bool ONE, int MOST>
void res_bwd(const ResProblem &p, int vec, dim3 grid, dim3 block, cudaStream_t stream) {
  const size_t smem = ONE ? block.y * 3 * 256 * sizeof(float) : 0;
  if (vec) gdp_res_bwd_kernel<T, true, ONE, MOST><<<grid, block, smem, stream>>>(p);
  else gdp_res_bwd_kernel<T, false, ONE, MOST><<<grid, block, smem, stream>>>(p);
}
template <typename T>
cudaError_t launch_res_bwd(const ResProblem &p, int vec, int64_t ctas, cudaStream_t stream) {
  const dim3 block(res_threads(p.C), res_rows(p.C)), grid((unsigned)ctas);
  if (block.y > 1) res_bwd<T, true, 128>(p, vec, grid, block, stream);
  else if (block.x <= 512) res_bwd<T, false, 512>(p, vec, grid, block, stream);
  else res_bwd<T, false, 1024>(p, vec, grid, block, stream);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace gdp
