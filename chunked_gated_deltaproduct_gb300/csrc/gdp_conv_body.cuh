// gdp_conv_body.cuh -- the short causal convolution's kernels, instantiated by type in gdp_conv_*.cu.
//
// A thread owns a vector of channels over a run of consecutive packed rows and keeps the last W - 1 inputs in
// registers, so that every row is read once (a run's first W - 1 rows twice).  Where a sequence begins, the
// window is that of its incoming state.
#pragma once

#include "gdp_conv.cuh"

namespace gdp {
namespace layer {

constexpr int kConvRun = 16;  // rows of a forward run
constexpr int kConvAhead = 8; // rows whose loads are under way at once

// x_{t-1-k} of sequence [b, ...) in win[k], from the incoming state where the row lies before b.
template <typename T, int V, int K>
__device__ __forceinline__ void load_window(const ConvProblem &p, int64_t t, int64_t b, const T *state, int64_t c, float (&win)[K][V]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t row = t - 1 - k;
    const T *at = row >= b ? static_cast<const T *>(p.x) + row * p.x_st + c : state ? state + (K + row - b) * p.C + c : nullptr;
#pragma unroll
    for (int i = 0; i < V; ++i) win[k][i] = 0.f;
    if (at) {
      const Vec<T, V> v = load_vec<T, V>(at);
#pragma unroll
      for (int i = 0; i < V; ++i) win[k][i] = to_f32(v.v[i]);
    }
  }
}
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvProblem &p, int64_t c, float (&w)[W][V], float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = p.w[(c + i) * W + j];
    b[i] = p.b ? p.b[c + i] : 0.f;
  }
}
// p_t of one row: taps oldest first.
template <int V, int W>
__device__ __forceinline__ void convolve(const float (&w)[W][V], const float (&b)[V], const float (&win)[W - 1][V], const float (&x)[V],
                                         float (&y)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float s = b[i];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][i], win[W - 2 - j][i], s);
    y[i] = fmaf(w[W - 1][i], x[i], s);
  }
}
template <int V, int K>
__device__ __forceinline__ void push_window(float (&win)[K][V], const float (&x)[V]) {
#pragma unroll
  for (int k = K - 1; k > 0; --k)
#pragma unroll
    for (int i = 0; i < V; ++i) win[k][i] = win[k - 1][i];
#pragma unroll
  for (int i = 0; i < V; ++i) win[0][i] = x[i];
}

// Final state of sequence i: the last K rows of the incoming state and the sequence's rows.  All are read before any is
// written (the cache is updated in place).
template <typename T, int V, int K>
__device__ __forceinline__ void final_state(const ConvProblem &p, int64_t i, int64_t c) {
  const T *src;
  T *dst;
  state_of<T>(p.s, i, K * p.C, p.p.status, false, &src, &dst);
  if (!dst) return;
  int64_t b, e;
  seq_rows(p.p, i, &b, &e);
  Vec<T, V> v[K];
#pragma unroll
  for (int r = 0; r < K; ++r) {
    const int64_t row = e - K + r;
    const T *at = row >= b ? static_cast<const T *>(p.x) + row * p.x_st + c : src ? src + (K + row - b) * p.C + c : nullptr;
    if (at) v[r] = load_vec<T, V>(at);
    else
#pragma unroll
      for (int k = 0; k < V; ++k) v[r].v[k] = from_f32<T>(0.f);
  }
#pragma unroll
  for (int r = 0; r < K; ++r) *reinterpret_cast<Vec<T, V> *>(dst + r * p.C + c) = v[r];
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) gdp_conv_fwd_kernel(const ConvProblem p) {
  constexpr int K = W - 1;
  const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_packed(p.p);
  if (c >= p.C) return;
  if (blockIdx.x >= p.runs) {  // states that are not updated in place
    const int64_t i = (blockIdx.x - p.runs) * blockDim.y + threadIdx.y;
    if (i < p.p.N) final_state<T, V, K>(p, i, c);
    return;
  }
  int64_t t = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * kConvRun;
  const int64_t stop = min(t + kConvRun, p.p.T);
  if (t >= stop) return;
  float w[W][V], bias[V], win[K][V];
  load_taps<V, W>(p, c, w, bias);
  const T *x_at = static_cast<const T *>(p.x) + c;
  T *y_at = static_cast<T *>(p.y) + c;
  int64_t i = seq_of_row(p.p, t), b, e;
  seq_rows(p.p, i, &b, &e);
  bool fresh = true;  // the window is not that of row t
  while (t < stop) {
    Vec<T, V> rows[kConvAhead];
#pragma unroll
    for (int k = 0; k < kConvAhead; ++k)
      if (t + k < stop) rows[k] = load_vec<T, V>(x_at + (t + k) * p.x_st);
#pragma unroll
    for (int k = 0; k < kConvAhead; ++k) {
      const int64_t row = t + k;
      if (row >= stop) break;
      if (row >= e) {
        while (row >= e && i + 1 < p.p.N) {
          ++i;
          seq_rows(p.p, i, &b, &e);
        }
        fresh = true;
      }
      if (row >= e || row < b) {  // padding (or a row that no bounds hold)
        if (p.zero_pad) {
          float zero[V] = {};
          store_vec<T, V>(y_at + row * p.C, zero);
        }
        continue;
      }
      if (fresh) {
        const T *src;
        T *dst;
        state_of<T>(p.s, i, K * p.C, p.p.status, c == 0, &src, &dst);
        load_window<T, V, K>(p, row, b, src, c, win);
        fresh = false;
      }
      float x[V], y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = to_f32(rows[k].v[j]);
      convolve<V, W>(w, bias, win, x, y);
      if (p.act == GDP_ACT_SILU)
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] *= sigmoid_fast(y[j]);
      store_vec<T, V>(y_at + row * p.C, y);
      push_window<V, K>(win, x);
    }
    t += kConvAhead;
  }
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) gdp_conv_states_kernel(const ConvProblem p) {
  const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V, i = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (c < p.C && i < p.p.N) final_state<T, V, W - 1>(p, i, c);
}

// One token per sequence: every value is touched once.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) gdp_conv_step_kernel(const ConvProblem p) {
  constexpr int K = W - 1;
  const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V, i = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (c >= p.C || i >= p.p.N) return;
  const T *src;
  T *dst;
  const Vec<T, V> now = load_vec<T, V>(static_cast<const T *>(p.x) + i * p.x_st + c);
  float w[W][V], bias[V], x[V], y[V], win[K][V];
  load_taps<V, W>(p, c, w, bias);
  state_of<T>(p.s, i, K * p.C, p.p.status, c == 0, &src, &dst);
  Vec<T, V> old[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (src) old[k] = load_vec<T, V>(src + k * p.C + c);
    else
#pragma unroll
      for (int j = 0; j < V; ++j) old[k].v[j] = from_f32<T>(0.f);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = to_f32(now.v[j]);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) win[K - 1 - k][j] = to_f32(old[k].v[j]);
  convolve<V, W>(w, bias, win, x, y);
  if (p.act == GDP_ACT_SILU)
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] *= sigmoid_fast(y[j]);
  store_vec<T, V>(static_cast<T *>(p.y) + i * p.C + c, y);
  if (dst) {
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) *reinterpret_cast<Vec<T, V> *>(dst + k * p.C + c) = old[k + 1];
    *reinterpret_cast<Vec<T, V> *>(dst + (K - 1) * p.C + c) = now;
  }
}

// dp = dy act'(p)
__device__ __forceinline__ float act_slope(float p, int act) {
  if (act != GDP_ACT_SILU) return 1.f;
  const float q = sigmoid_fast(p);
  return q * fmaf(p, 1.f - q, 1.f);
}

// d_initial_state of sequence i: what its first K outputs (and, where it is shorter, its final state) pass back.
template <typename T, int W, int V>
__device__ __forceinline__ void initial_gradient(const ConvProblem &p, int64_t i, int64_t c) {
  constexpr int K = W - 1;
  int64_t b, e;
  seq_rows(p.p, i, &b, &e);
  const T *state = p.s.init ? static_cast<const T *>(p.s.init) + i * K * p.C : nullptr;
  float w[W][V], bias[V], win[K][V], d[K][V] = {};
  load_taps<V, W>(p, c, w, bias);
  load_window<T, V, K>(p, b, b, state, c, win);
#pragma unroll
  for (int k = 0; k < K; ++k) {  // row b + k
    if (b + k >= e) {            // the sequence has k rows: incoming rows k .. K - 1 are final ones 0 .. K - 1 - k
      if (p.dfin && b + k == e)
#pragma unroll
        for (int r = 0; r + k < K; ++r) {
          const Vec<T, V> f = load_vec<T, V>(static_cast<const T *>(p.dfin) + (i * K + r) * p.C + c);
#pragma unroll
          for (int j = 0; j < V; ++j) d[k + r][j] += to_f32(f.v[j]);
        }
      continue;
    }
    const Vec<T, V> xr = load_vec<T, V>(static_cast<const T *>(p.x) + (b + k) * p.x_st + c),
                    dr = load_vec<T, V>(static_cast<const T *>(p.dy) + (b + k) * p.dy_st + c);
    float x[V], y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = to_f32(xr.v[j]);
    convolve<V, W>(w, bias, win, x, y);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float dp = to_f32(dr.v[j]) * act_slope(y[j], p.act);
#pragma unroll
      for (int r = 0; r < K; ++r)
        if (r >= k) d[r][j] = fmaf(w[r - k >= 0 ? r - k : 0][j], dp, d[r][j]);
    }
    push_window<V, K>(win, x);
  }
  T *out = static_cast<T *>(p.dinit) + i * K * p.C + c;
#pragma unroll
  for (int r = 0; r < K; ++r) store_vec<T, V>(out + r * p.C, d[r]);
}

// A part is a run of rows [t0, t1).  A thread walks it in order and K rows beyond, forms p again from its window of
// inputs, and holds the unfinished input gradients of the last K rows in registers; the weights' sums over the
// part stay in registers too and leave once.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) gdp_conv_bwd_kernel(const ConvProblem p) {
  constexpr int K = W - 1, A = 4;  // rows whose loads are under way at once
  const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_packed(p.p);
  if (c >= p.C) return;
  if (blockIdx.x >= p.runs) {
    const int64_t i = (blockIdx.x - p.runs) * blockDim.y + threadIdx.y;
    if (i < p.p.N) initial_gradient<T, W, V>(p, i, c);
    return;
  }
  const int64_t part = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t t0 = min(part * p.part_rows, p.p.T), t1 = min(t0 + p.part_rows, p.p.T), last = min(t1 + K, p.p.T);
  float w[W][V], bias[V], win[K][V], pend[K][V], dw[W][V] = {}, db[V] = {};
  const T *x_at = static_cast<const T *>(p.x) + c, *dy_at = static_cast<const T *>(p.dy) + c;
  T *dx_at = static_cast<T *>(p.dx) + c;
  if (t0 < t1) {
    load_taps<V, W>(p, c, w, bias);
    int64_t i = seq_of_row(p.p, t0), b, e;
    seq_rows(p.p, i, &b, &e);
    bool fresh = true, done = false;
    // The sequence ends before row t: its last rows' gradients are complete but for the final state's.
    auto flush = [&](int64_t t) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int64_t row = t - 1 - k;
        if (row < b || row < t0 || row >= t1) continue;
        if (p.dfin) {
          const Vec<T, V> f = load_vec<T, V>(static_cast<const T *>(p.dfin) + (i * K + (K - 1 - k)) * p.C + c);
#pragma unroll
          for (int j = 0; j < V; ++j) pend[k][j] += to_f32(f.v[j]);
        }
        store_vec<T, V>(dx_at + row * p.C, pend[k]);
      }
    };
    for (int64_t t = t0; t < last && !done; t += A) {
      Vec<T, V> xs[A], ds[A];
#pragma unroll
      for (int k = 0; k < A; ++k)
        if (t + k < last) {
          xs[k] = load_vec<T, V>(x_at + (t + k) * p.x_st);
          ds[k] = load_vec<T, V>(dy_at + (t + k) * p.dy_st);
        }
#pragma unroll
      for (int k = 0; k < A; ++k) {
        const int64_t row = t + k;
        if (row >= last || done) break;
        if (row >= e) {
          if (!fresh) flush(row);
          fresh = true;
          if (row >= t1) {
            done = true;
            break;
          }
          while (row >= e && i + 1 < p.p.N) {
            ++i;
            seq_rows(p.p, i, &b, &e);
          }
        }
        if (row >= e || row < b) {
          if (row < t1) {
            float zero[V] = {};
            store_vec<T, V>(dx_at + row * p.C, zero);
          }
          continue;
        }
        if (fresh) {
          const T *state = p.s.init ? static_cast<const T *>(p.s.init) + i * K * p.C : nullptr;
          load_window<T, V, K>(p, row, b, state, c, win);
#pragma unroll
          for (int r = 0; r < K; ++r)
#pragma unroll
            for (int j = 0; j < V; ++j) pend[r][j] = 0.f;
          fresh = false;
        }
        float x[V], y[V], dp[V], out[V];
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = to_f32(xs[k].v[j]);
        convolve<V, W>(w, bias, win, x, y);
        const float own = row < t1 ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          dp[j] = to_f32(ds[k].v[j]) * act_slope(y[j], p.act);
          out[j] = fmaf(w[0][j], dp[j], pend[K - 1][j]);
#pragma unroll
          for (int r = K - 1; r > 0; --r) pend[r][j] = fmaf(w[K - r][j], dp[j], pend[r - 1][j]);
          pend[0][j] = w[K][j] * dp[j];
        }
        if (own != 0.f) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            db[j] += dp[j];
            dw[K][j] = fmaf(dp[j], x[j], dw[K][j]);
#pragma unroll
            for (int r = 0; r < K; ++r) dw[r][j] = fmaf(dp[j], win[K - 1 - r][j], dw[r][j]);
          }
        }
        if (row - K >= b && row - K >= t0) store_vec<T, V>(dx_at + (row - K) * p.C, out);
        push_window<V, K>(win, x);
      }
    }
    // the tensors end here, and the sequence with them
    if (!done && !fresh && last == p.p.T && e == last && last < t1 + K) flush(last);
  }
  float *to = p.partial + part * (W + 1) * p.C + c;
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int r = 0; r < W; ++r) to[r * p.C + j] = dw[r][j];
    to[W * p.C + j] = db[j];
  }
}

template <typename T, int V>
cudaError_t conv_fwd(ConvProblem &p, int width, bool states, cudaStream_t stream) {
  const int64_t vecs = (p.C + V - 1) / V;
  const dim3 block = conv_block(vecs);
  p.runs = (p.p.T + kConvRun * block.y - 1) / (kConvRun * block.y);
  const dim3 grid((unsigned)(p.runs + (states ? (p.p.N + block.y - 1) / block.y : 0)), (unsigned)((vecs + block.x - 1) / block.x));
  if (grid.x == 0) return cudaSuccess;
  if (width == 2) gdp_conv_fwd_kernel<T, 2, V><<<grid, block, 0, stream>>>(p);
  else if (width == 3) gdp_conv_fwd_kernel<T, 3, V><<<grid, block, 0, stream>>>(p);
  else gdp_conv_fwd_kernel<T, 4, V><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_conv_fwd(ConvProblem &p, int width, int vec, bool states, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  if (vec == V) return conv_fwd<T, V>(p, width, states, stream);
  return vec >= 2 ? conv_fwd<T, 2>(p, width, states, stream) : conv_fwd<T, 1>(p, width, states, stream);
}

template <typename T>
cudaError_t launch_conv_states(const ConvProblem &p, int width, cudaStream_t stream) {
  const dim3 block = conv_block(p.C);
  const dim3 grid((unsigned)((p.p.N + block.y - 1) / block.y), (unsigned)((p.C + block.x - 1) / block.x));
  if (width == 2) gdp_conv_states_kernel<T, 2, 1><<<grid, block, 0, stream>>>(p);
  else if (width == 3) gdp_conv_states_kernel<T, 3, 1><<<grid, block, 0, stream>>>(p);
  else gdp_conv_states_kernel<T, 4, 1><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_conv_step(const ConvProblem &p, int width, cudaStream_t stream) {
  const dim3 block = conv_block(p.C);
  const dim3 grid((unsigned)((p.p.N + block.y - 1) / block.y), (unsigned)((p.C + block.x - 1) / block.x));
  if (width == 2) gdp_conv_step_kernel<T, 2, 1><<<grid, block, 0, stream>>>(p);
  else if (width == 3) gdp_conv_step_kernel<T, 3, 1><<<grid, block, 0, stream>>>(p);
  else gdp_conv_step_kernel<T, 4, 1><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t conv_bwd(ConvProblem &p, int width, cudaStream_t stream) {
  const int64_t vecs = (p.C + V - 1) / V;
  const dim3 block = conv_block(vecs);
  p.parts = conv_parts(p.p.T, vecs, sm_count());
  p.part_rows = (p.p.T + p.parts - 1) / p.parts;
  p.runs = p.parts / block.y;
  const dim3 grid((unsigned)(p.runs + (p.dinit ? (p.p.N + block.y - 1) / block.y : 0)), (unsigned)((vecs + block.x - 1) / block.x));
  if (width == 2) gdp_conv_bwd_kernel<T, 2, V><<<grid, block, 0, stream>>>(p);
  else if (width == 3) gdp_conv_bwd_kernel<T, 3, V><<<grid, block, 0, stream>>>(p);
  else gdp_conv_bwd_kernel<T, 4, V><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_conv_bwd(ConvProblem &p, int width, int vec, cudaStream_t stream) {
  if (vec >= 4) return conv_bwd<T, 4>(p, width, stream);
  return vec >= 2 ? conv_bwd<T, 2>(p, width, stream) : conv_bwd<T, 1>(p, width, stream);
}

}  // namespace layer
}  // namespace gdp
