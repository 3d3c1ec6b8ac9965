// gdp_conv_body.cuh -- the short causal convolution's kernels, instantiated by type in gdp_conv_*.cu.
//
// A thread owns a vector of channels over a run of consecutive packed rows and keeps the last W - 1 inputs in
// registers, so that every row is read once (a run's first W - 1 rows twice).  Where a sequence begins, the
// window is that of its incoming state.
//
// 65536 x 4096 bf16, 4 taps, SiLU: forward 168 us, 6.35 TB/s, bound by memory (rows asked for only when they are needed: 389 us;
// by a double buffer of registers: 389 too); backward 315 us, 5.1 TB/s, bound by the latency of 77 instructions a row and thread at
// 16 warps per SM; f16 172 and 332 (with the column sums), 32768 rows of fp32 166 and 284.  One token for 64 x 4096: 2.9 us on the
// device, a launch's latency and three loads' behind one another (512 x 4096: 15 us a call).
#pragma once

#include "gdp_conv.cuh"

namespace gdp {
namespace layer {

constexpr int kConvAhead = 4; // rows that are worked on together
constexpr int kConvSums = 64;  // rows whose products a sum of the backward pass takes in registers

// Rows on their way to a thread, S tensors, kConvAhead rows a batch.  Asynchronous copies into places of shared memory
// that are the thread's own (no barriers) keep two batches under way without registers; values below the copies' least
// size (four bytes) wait in registers, one batch ahead.
template <typename R, int S>
struct RowQueue {
  static constexpr bool ASYNC = sizeof(R) >= 4;
  static constexpr int A = kConvAhead, DEEP = ASYNC ? 2 : 1, BYTES = ASYNC ? 3 * A * S * kConvThreads * (int)sizeof(R) : 16;
  R *own;
  R now[ASYNC ? 1 : S * A], next[ASYNC ? 1 : S * A];
  __device__ __forceinline__ explicit RowQueue(unsigned char *smem)
      : own(reinterpret_cast<R *>(smem) + threadIdx.y * blockDim.x + threadIdx.x) {}
  // row k of tensor s of the batch in place `at` (0, 1, 2 in turn); every batch is asked for in order, and closed
  __device__ __forceinline__ void ask(int at, int s, int k, const void *from) {
    if constexpr (ASYNC) {
      const uint32_t to = sm100::smem_u32(own + ((at * A + k) * S + s) * kConvThreads);
      if constexpr (sizeof(R) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
      else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"((int)sizeof(R)) : "memory");
    } else {
      next[s * A + k] = *static_cast<const R *>(from);
    }
  }
  __device__ __forceinline__ void close() {
    if constexpr (ASYNC) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void wait() {  // before `ask` of the batch DEEP further on
    if constexpr (ASYNC) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
#pragma unroll
      for (int k = 0; k < S * A; ++k) now[k] = next[k];
  }
  __device__ __forceinline__ R get(int at, int s, int k) const {
    if constexpr (ASYNC) return own[((at * A + k) * S + s) * kConvThreads];
    else return now[s * A + k];
  }
};

// V channels as pairs in fp32 (one channel: a pair whose second value is none).
template <int V>
struct Pairs {
  static constexpr int N = V > 1 ? V / 2 : 1;
  float2 v[N];
};
template <typename T, int V>
__device__ __forceinline__ Pairs<V> pairs_of(const Vec<T, V> &r) {
  Pairs<V> o;
  if constexpr (V == 1) o.v[0] = make_float2(to_f32(r.v[0]), 0.f);
  else
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      if constexpr (sizeof(T) == 4) o.v[k] = make_float2(r.v[2 * k], r.v[2 * k + 1]);
      else o.v[k] = widen<T>(reinterpret_cast<const uint32_t *>(r.v)[k]);
    }
  return o;
}
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T *at, const Pairs<V> &p) {
  Vec<T, V> o;
  if constexpr (V == 1) o.v[0] = from_f32<T>(p.v[0].x);
  else
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      if constexpr (sizeof(T) == 4) o.v[2 * k] = p.v[k].x, o.v[2 * k + 1] = p.v[k].y;
      else reinterpret_cast<uint32_t *>(o.v)[k] = narrow<T>(p.v[k]);
    }
  *reinterpret_cast<Vec<T, V> *>(at) = o;
}
template <int V>
__device__ __forceinline__ Pairs<V> no_pairs() {
  Pairs<V> o;
#pragma unroll
  for (int k = 0; k < Pairs<V>::N; ++k) o.v[k] = make_float2(0.f, 0.f);
  return o;
}

// x_{t-1-k} of sequence [b, ...) in win[k], from the incoming state where the row lies before b.
template <typename T, int V, int K>
__device__ __forceinline__ void load_window(const ConvProblem &p, int64_t t, int64_t b, const T *state, int64_t c, Pairs<V> (&win)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t row = t - 1 - k;
    const T *at = row >= b ? static_cast<const T *>(p.x) + row * p.x_st + c : state ? state + (K + row - b) * p.C + c : nullptr;
    win[k] = at ? pairs_of<T, V>(load_vec<T, V>(at)) : no_pairs<V>();
  }
}
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvProblem &p, int64_t c, Pairs<V> (&w)[W], Pairs<V> &b) {
  b = no_pairs<V>();
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = no_pairs<V>();
  float taps[V * W];
  if (p.quad_taps && V * W % 4 == 0) {
#pragma unroll
    for (int k = 0; k < V * W / 4; ++k) {
      const float4 q = reinterpret_cast<const float4 *>(p.w + c * W)[k];
      taps[4 * k] = q.x, taps[4 * k + 1] = q.y, taps[4 * k + 2] = q.z, taps[4 * k + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V * W; ++k) taps[k] = p.w[c * W + k];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) (i % 2 ? w[j].v[i / 2].y : w[j].v[i / 2].x) = taps[i * W + j];
    if (p.b) (i % 2 ? b.v[i / 2].y : b.v[i / 2].x) = p.b[c + i];
  }
}
// p_t of one row: taps oldest first.
template <int V, int W>
__device__ __forceinline__ Pairs<V> convolve(const Pairs<V> (&w)[W], const Pairs<V> &b, const Pairs<V> (&win)[W - 1], const Pairs<V> &x) {
  Pairs<V> y;
#pragma unroll
  for (int i = 0; i < Pairs<V>::N; ++i) {
    float2 s = b.v[i];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = fma2(w[j].v[i], win[W - 2 - j].v[i], s);
    y.v[i] = fma2(w[W - 1].v[i], x.v[i], s);
  }
  return y;
}
template <int V, int K>
__device__ __forceinline__ void push_window(Pairs<V> (&win)[K], const Pairs<V> &x) {
#pragma unroll
  for (int k = K - 1; k > 0; --k) win[k] = win[k - 1];
  win[0] = x;
}
template <int V>
__device__ __forceinline__ void activate(Pairs<V> &y) {
#pragma unroll
  for (int i = 0; i < Pairs<V>::N; ++i) y.v[i] = mul2(y.v[i], sigmoid2(y.v[i]));
}

// Final state of sequence i: the last K rows of the incoming state and the sequence's rows.  All are read before any is
// written (the cache is updated in place).
template <typename T, int V, int K>
__device__ __forceinline__ void final_state(const ConvProblem &p, int64_t i, int64_t c) {  // (reports bad slots, an empty sequence's too)
  const T *src;
  T *dst;
  state_of<T>(p.s, i, K * p.C, p.p.status, c == 0, &src, &dst);
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
  constexpr int K = W - 1, A = kConvAhead;
  const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_packed(p.p);
  if (c >= p.C) return;
  if (blockIdx.x >= p.runs) {  // states that are not updated in place
    const int64_t i = (blockIdx.x - p.runs) * blockDim.y + threadIdx.y;
    if (i < p.p.N) final_state<T, V, K>(p, i, c);
    return;
  }
  const int64_t t0 = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * p.run, stop = min(t0 + p.run, p.p.T);
  if (t0 >= stop) return;
  const T *x_at = static_cast<const T *>(p.x) + c;
  T *y_at = static_cast<T *>(p.y) + c;
  using Queue = RowQueue<Vec<T, V>, 1>;
  __shared__ __align__(16) unsigned char room[Queue::BYTES];
  Queue queue(room);
  int left = (int)(stop - t0);  // rows still to be asked for
  const T *from = x_at + t0 * p.x_st;
  auto ask = [&](int at) {
#pragma unroll
    for (int k = 0; k < A; ++k)
      if (k < left) queue.ask(at, 0, k, from + k * p.x_st);
    left -= A;
    from += A * p.x_st;
    queue.close();
  };
#pragma unroll
  for (int n = 0; n < Queue::DEEP; ++n) ask(n);
  Pairs<V> w[W], bias, win[K];
  load_taps<V, W>(p, c, w, bias);
  int64_t i = seq_of_row(p.p, t0), b, e;
  seq_rows(p.p, i, &b, &e);
  bool fresh = true;  // the window is not that of the row
  auto enter = [&](int64_t row) {
    const T *src;
    T *dst;
    state_of<T>(p.s, i, K * p.C, p.p.status, c == 0, &src, &dst);
    load_window<T, V, K>(p, row, b, src, c, win);
    fresh = false;
  };
  auto one = [&](T *to, const Vec<T, V> &raw) {
    const Pairs<V> x = pairs_of<T, V>(raw);
    Pairs<V> y = convolve<V, W>(w, bias, win, x);
    if (p.act == GDP_ACT_SILU) activate<V>(y);
    store_pairs<T, V>(to, y);
    push_window<V, K>(win, x);
  };
  T *to = y_at + t0 * p.C;
  int at = 0;
  for (int64_t t = t0; t < stop; t += A, to += A * p.C, at = at == 2 ? 0 : at + 1) {
    queue.wait();
    ask(at + Queue::DEEP < 3 ? at + Queue::DEEP : at + Queue::DEEP - 3);
    if (t >= b && t + A <= min(e, stop)) {  // all of one sequence
      if (fresh) enter(t);
#pragma unroll
      for (int k = 0; k < A; ++k) one(to + k * p.C, queue.get(at, 0, k));
    } else {
#pragma unroll
      for (int k = 0; k < A; ++k) {
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
          if (p.zero_pad) store_pairs<T, V>(to + k * p.C, no_pairs<V>());
          continue;
        }
        if (fresh) enter(row);
        one(to + k * p.C, queue.get(at, 0, k));
      }
    }
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
  Pairs<V> w[W], bias, win[K];
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
  for (int k = 0; k < K; ++k) win[K - 1 - k] = pairs_of<T, V>(old[k]);
  Pairs<V> y = convolve<V, W>(w, bias, win, pairs_of<T, V>(now));
  if (p.act == GDP_ACT_SILU) activate<V>(y);
  store_pairs<T, V>(static_cast<T *>(p.y) + i * p.C + c, y);
  if (dst) {
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) *reinterpret_cast<Vec<T, V> *>(dst + k * p.C + c) = old[k + 1];
    *reinterpret_cast<Vec<T, V> *>(dst + (K - 1) * p.C + c) = now;
  }
}

// dp = dy act'(p)
template <int V>
__device__ __forceinline__ Pairs<V> through_act(const Pairs<V> &p, const Pairs<V> &dy, int act) {
  if (act != GDP_ACT_SILU) return dy;
  Pairs<V> o;
#pragma unroll
  for (int i = 0; i < Pairs<V>::N; ++i) {
    const float2 q = sigmoid2(p.v[i]);
    const float2 rest = fma2(q, both(-1.f), both(1.f));
    o.v[i] = mul2(dy.v[i], mul2(q, fma2(p.v[i], rest, both(1.f))));
  }
  return o;
}

// d_initial_state of sequence i: what its first K outputs (and, where it is shorter, its final state) pass back.
template <typename T, int W, int V>
__device__ __forceinline__ void initial_gradient(const ConvProblem &p, int64_t i, int64_t c) {
  constexpr int K = W - 1, N = Pairs<V>::N;
  int64_t b, e;
  seq_rows(p.p, i, &b, &e);
  const T *state = p.s.init ? static_cast<const T *>(p.s.init) + i * K * p.C : nullptr;
  Pairs<V> w[W], bias, win[K], d[K];
  load_taps<V, W>(p, c, w, bias);
  load_window<T, V, K>(p, b, b, state, c, win);
#pragma unroll
  for (int k = 0; k < K; ++k) d[k] = no_pairs<V>();
#pragma unroll
  for (int k = 0; k < K; ++k) {  // row b + k
    if (b + k >= e) {            // the sequence has k rows: incoming rows k .. K - 1 are final ones 0 .. K - 1 - k
      if (p.dfin && b + k == e)
#pragma unroll
        for (int r = 0; r + k < K; ++r) {
          const Pairs<V> f = pairs_of<T, V>(load_vec<T, V>(static_cast<const T *>(p.dfin) + (i * K + r) * p.C + c));
#pragma unroll
          for (int j = 0; j < N; ++j) d[k + r].v[j] = add2(d[k + r].v[j], f.v[j]);
        }
      continue;
    }
    const Pairs<V> x = pairs_of<T, V>(load_vec<T, V>(static_cast<const T *>(p.x) + (b + k) * p.x_st + c));
    const Pairs<V> g = pairs_of<T, V>(load_vec<T, V>(static_cast<const T *>(p.dy) + (b + k) * p.dy_st + c));
    const Pairs<V> dp = through_act<V>(convolve<V, W>(w, bias, win, x), g, p.act);
#pragma unroll
    for (int r = 0; r < K; ++r)
      if (r >= k)
#pragma unroll
        for (int j = 0; j < N; ++j) d[r].v[j] = fma2(w[r >= k ? r - k : 0].v[j], dp.v[j], d[r].v[j]);
    push_window<V, K>(win, x);
  }
  T *out = static_cast<T *>(p.dinit) + i * K * p.C + c;
#pragma unroll
  for (int r = 0; r < K; ++r) store_pairs<T, V>(out + r * p.C, d[r]);
}

// A part is a run of rows [t0, t1).  A thread walks it in order and K rows beyond, forms p again from its window of
// inputs, and holds the unfinished input gradients of the last K rows in registers.  The weights' sums run in two steps, so that
// their roundings grow with kConvSums rows and not with a part's (65536 x 4096, error of dweight: 5.4e-7 to 2.1e-7; the parts of
// odd widths are four times as long): in registers, and from there into the thread's place of shared memory.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) gdp_conv_bwd_kernel(const ConvProblem p) {
  constexpr int K = W - 1, N = Pairs<V>::N, A = kConvAhead;
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
  Pairs<V> w[W], bias, win[K], pend[K], dw[W], db = no_pairs<V>();
  __shared__ float2 sums[(W + 1) * N][kConvThreads];
  float2 *own_sums = &sums[0][threadIdx.y * blockDim.x + threadIdx.x];
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j] = no_pairs<V>();
#pragma unroll
  for (int k = 0; k < (W + 1) * N; ++k) own_sums[k * kConvThreads] = make_float2(0.f, 0.f);
  auto add_up = [&] {
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int r = 0; r < W; ++r) own_sums[(r * N + j) * kConvThreads] = add2(own_sums[(r * N + j) * kConvThreads], dw[r].v[j]);
      own_sums[(W * N + j) * kConvThreads] = add2(own_sums[(W * N + j) * kConvThreads], db.v[j]);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j] = no_pairs<V>();
    db = no_pairs<V>();
  };
  const T *x_at = static_cast<const T *>(p.x) + c, *dy_at = static_cast<const T *>(p.dy) + c;
  T *dx_at = static_cast<T *>(p.dx) + c;
  if (t0 < t1) {
    using Queue = RowQueue<Vec<T, V>, 2>;
    __shared__ __align__(16) unsigned char room[Queue::BYTES];
    Queue queue(room);
    int left = (int)(last - t0);  // rows still to be asked for
    const T *x_from = x_at + t0 * p.x_st, *dy_from = dy_at + t0 * p.dy_st;
    auto ask = [&](int at) {
#pragma unroll
      for (int k = 0; k < A; ++k)
        if (k < left) {
          queue.ask(at, 0, k, x_from + k * p.x_st);
          queue.ask(at, 1, k, dy_from + k * p.dy_st);
        }
      left -= A;
      x_from += A * p.x_st;
      dy_from += A * p.dy_st;
      queue.close();
    };
#pragma unroll
    for (int n = 0; n < Queue::DEEP; ++n) ask(n);
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
          const Pairs<V> f = pairs_of<T, V>(load_vec<T, V>(static_cast<const T *>(p.dfin) + (i * K + (K - 1 - k)) * p.C + c));
#pragma unroll
          for (int j = 0; j < N; ++j) pend[k].v[j] = add2(pend[k].v[j], f.v[j]);
        }
        store_pairs<T, V>(dx_at + row * p.C, pend[k]);
      }
    };
    auto enter = [&](int64_t row) {
      const T *state = p.s.init ? static_cast<const T *>(p.s.init) + i * K * p.C : nullptr;
      load_window<T, V, K>(p, row, b, state, c, win);
#pragma unroll
      for (int r = 0; r < K; ++r) pend[r] = no_pairs<V>();
      fresh = false;
    };
    // One row: `own`: it belongs to the part; the row K before it (at `before`) is complete then, and leaves with `out`.
    auto one = [&](T *before, const Vec<T, V> &xr, const Vec<T, V> &dr, bool own, bool out) {
      const Pairs<V> x = pairs_of<T, V>(xr), dp = through_act<V>(convolve<V, W>(w, bias, win, x), pairs_of<T, V>(dr), p.act);
      Pairs<V> ready;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        ready.v[j] = fma2(w[0].v[j], dp.v[j], pend[K - 1].v[j]);
#pragma unroll
        for (int r = K - 1; r > 0; --r) pend[r].v[j] = fma2(w[K - r].v[j], dp.v[j], pend[r - 1].v[j]);
        pend[0].v[j] = mul2(w[K].v[j], dp.v[j]);
      }
      if (own) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          db.v[j] = add2(db.v[j], dp.v[j]);
          dw[K].v[j] = fma2(dp.v[j], x.v[j], dw[K].v[j]);
#pragma unroll
          for (int r = 0; r < K; ++r) dw[r].v[j] = fma2(dp.v[j], win[K - 1 - r].v[j], dw[r].v[j]);
        }
      }
      if (out) store_pairs<T, V>(before, ready);
      push_window<V, K>(win, x);
    };
    T *before = dx_at + (t0 - K) * p.C;  // (written where it is a row of the part)
    int at = 0;
    for (int64_t t = t0, stop; t < last && !done; add_up()) {
      stop = min(t + kConvSums, last);
      for (; t < stop && !done; t += A, before += A * p.C, at = at == 2 ? 0 : at + 1) {
        queue.wait();
        ask(at + Queue::DEEP < 3 ? at + Queue::DEEP : at + Queue::DEEP - 3);
        if (!fresh && t - K >= max(t0, b) && t + A <= min(e, t1)) {  // all of one sequence and the part
#pragma unroll
          for (int k = 0; k < A; ++k) one(before + k * p.C, queue.get(at, 0, k), queue.get(at, 1, k), true, true);
        } else {
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
              if (row < t1) store_pairs<T, V>(dx_at + row * p.C, no_pairs<V>());
              continue;
            }
            if (fresh) enter(row);
            one(before + k * p.C, queue.get(at, 0, k), queue.get(at, 1, k), row < t1, row - K >= b && row - K >= t0);
          }
        }
      }
    }
    // the tensors end here, and the sequence with them
    if (!done && !fresh && last == p.p.T && e == last && last < t1 + K) flush(last);
    asm volatile("cp.async.wait_all;" ::: "memory");  // (rows of the next sequence, where this one ended first)
  }
  float *to = p.partial + part * (W + 1) * p.C + c;
#pragma unroll
  for (int r = 0; r <= W; ++r)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float2 v = own_sums[(r * N + j / 2) * kConvThreads];
      to[r * p.C + j] = j % 2 ? v.y : v.x;
    }
}

template <typename T, int V>
cudaError_t conv_fwd(ConvProblem &p, int width, bool states, cudaStream_t stream) {
  const int64_t vecs = (p.C + V - 1) / V;
  const dim3 block = conv_block(vecs);
  // short batches: sixteen rows a thread, so that there are enough of them; else 64, of which the first three are read twice
  const int64_t across = (vecs + block.x - 1) / block.x;
  p.run = p.p.T * across / (64 * block.y) >= 8 * sm_count() ? 64 : 16;
  p.runs = (p.p.T + p.run * block.y - 1) / (p.run * block.y);
  if (p.runs == 0) p.runs = 1;  // (the bounds are still checked)
  const dim3 grid((unsigned)(p.runs + (states ? (p.p.N + block.y - 1) / block.y : 0)), (unsigned)((vecs + block.x - 1) / block.x));
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
  p.runs = p.parts / block.y;  // (one at least: the bounds of no rows are checked too)
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
