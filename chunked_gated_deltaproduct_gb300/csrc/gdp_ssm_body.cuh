// gdp_ssm_body.cuh -- the selective state space scan's kernels, instantiated by type in gdp_ssm_*.cu.
//
// A channel's S states belong to L lanes of one warp, four each; a CTA takes 128 / L channels of one group along a
// whole sequence.  Per tile of tokens the CTA first forms what a (token, channel) pair needs once (step size e, e x) in
// shared memory, then every lane runs its states over the tile's tokens, then the outputs are finished pair by pair.
#pragma once

#include "gdp_ssm.cuh"

namespace gdp {
namespace layer {

constexpr int kSsmTile = 32;  // tokens of a forward tile
constexpr int kQ = 4;         // states of a lane

// Sums over the R lanes whose numbers differ by multiples of STRIDE, V values each: a lane of rank r ends up with values
// r V / R ... of the sums (with R >= V, value r V / R rounded down), in v[0 ...].
template <int V, int R, int STRIDE>
__device__ __forceinline__ void sum_scatter(float *v, int rank) {
  if constexpr (R > 1) {
    constexpr int H = R / 2;
    if constexpr (V > 1) {
      const bool up = rank & H;
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const float give = up ? v[k] : v[k + V / 2], keep = up ? v[k + V / 2] : v[k];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, give, H * STRIDE);
      }
      sum_scatter<V / 2, H, STRIDE>(v, rank & (H - 1));
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], H * STRIDE);
      sum_scatter<1, H, STRIDE>(v, rank & (H - 1));
    }
  }
}

// log(1 + e^v) = max(v, 0) + log(1 + w) with w = e^-|v| in (0, 1]; log(1 + w) = 2 artanh(s), s = w / (2 + w) <= 1/3, by
// its power series: what is left out is below s^17 / 17 < 2^-30, and small w keep their relative precision.
__device__ __forceinline__ float softplus(float v) {
  const float w = exp_fast(-fabsf(v));
  const float s = w * rcp(2.f + w), q = s * s;
  float r = fmaf(q, 1.f / 15.f, 1.f / 13.f);
  r = fmaf(q, r, 1.f / 11.f);
  r = fmaf(q, r, 1.f / 9.f);
  r = fmaf(q, r, 1.f / 7.f);
  r = fmaf(q, r, 1.f / 5.f);
  r = fmaf(q, r, 1.f / 3.f);
  r = fmaf(q, r, 1.f);
  return fmaxf(v, 0.f) + 2.f * s * r;
}

template <typename T>
__device__ __forceinline__ float load_step(const SsmProblem &p, int64_t t, int64_t c) {
  const float v = p.dt_f32 ? static_cast<const float *>(p.dt)[t * p.dt_st + c] : to_f32(static_cast<const T *>(p.dt)[t * p.dt_st + c]);
  return p.bias ? v + p.bias[c] : v;
}

// Four states of one channel from / to [C, S] rows; n of them exist.
__device__ __forceinline__ void load_states(const float *at, int n, int quad, float (&h)[kQ]) {
  if (quad) {
    const float4 v = n > 0 ? *reinterpret_cast<const float4 *>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
    h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
  } else {
#pragma unroll
    for (int k = 0; k < kQ; ++k) h[k] = k < n ? at[k] : 0.f;
  }
}
__device__ __forceinline__ void store_states(float *at, int n, int quad, const float (&h)[kQ]) {
  if (quad) {
    if (n > 0) *reinterpret_cast<float4 *>(at) = make_float4(h[0], h[1], h[2], h[3]);
  } else {
#pragma unroll
    for (int k = 0; k < kQ; ++k)
      if (k < n) at[k] = h[k];
  }
}

// Which channels and states a thread has.
template <int L>
struct SsmPlace {
  static constexpr int CH = kSsmThreads / L, SP = L * kQ;  // channels of a CTA, states with padding
  int64_t g, c0;  // group, the CTA's first channel
  int cn;         // the CTA's channels
  int ch, j, n;   // the thread's channel in the CTA, lane of the channel, states that exist
  int64_t c;
  __device__ __forceinline__ SsmPlace(const SsmProblem &p, int64_t tile) {
    g = tile / p.tiles;
    c0 = g * p.per + (tile % p.tiles) * CH;
    cn = (int)min((int64_t)CH, (g + 1) * p.per - c0);
    ch = threadIdx.x / L;
    j = threadIdx.x % L;
    n = ch < cn ? max(0, min(kQ, (int)p.S - j * kQ)) : 0;
    c = c0 + ch;
  }
};

// Zeros into rows [cu_seqlens[N], T) of a [T, C] output, the CTA's channels.
template <typename T>
__device__ __forceinline__ void zero_tail(const SsmProblem &p, T *out, int64_t c0, int cn) {
  if (!out) return;
  for (int64_t t = cu_at(p.p, p.p.N) + threadIdx.x / 32; t < p.p.T; t += kSsmThreads / 32)
    for (int c = threadIdx.x % 32; c < cn; c += 32) out[t * p.C + c0 + c] = from_f32<T>(0.f);
}

// B and C of a tile's tokens in fp32, padded states as zeros.
template <typename T, int SP>
__device__ __forceinline__ void load_vectors(const SsmProblem &p, int64_t g, int64_t row, int rows, float (*B)[SP], float (*Cm)[SP]) {
  for (int i = threadIdx.x; i < rows * SP; i += kSsmThreads) {
    const int t = i / SP, s = i % SP;
    B[t][s] = s < p.S ? to_f32(static_cast<const T *>(p.B)[(row + t) * p.B_st + g * p.B_sg + s]) : 0.f;
    Cm[t][s] = s < p.S ? to_f32(static_cast<const T *>(p.Cm)[(row + t) * p.C_st + g * p.C_sg + s]) : 0.f;
  }
}

template <typename T, int L>
__global__ void __launch_bounds__(kSsmThreads) gdp_ssm_fwd_kernel(const SsmProblem p) {
  using Place = SsmPlace<L>;
  constexpr int CH = Place::CH, SP = Place::SP, PAIRS = kSsmTile * CH / kSsmThreads;
  __shared__ float2 steps[kSsmTile][CH];  // e, e x
  __shared__ __align__(16) float Bs[kSsmTile][SP], Cs[kSsmTile][SP];
  __shared__ float ys[kSsmTile][CH];
  const Place at(p, blockIdx.y);
  if (blockIdx.x == 0 && blockIdx.y == 0) check_packed(p.p);
  if (blockIdx.x == p.p.N) {
    zero_tail<T>(p, static_cast<T *>(p.y), at.c0, at.cn);
    return;
  }
  const int64_t i = blockIdx.x;
  int64_t b, e;
  seq_rows(p.p, i, &b, &e);
  const float *src;
  float *dst;
  state_of<float>(p.s, i, p.C * p.S, p.p.status, threadIdx.x == 0 && blockIdx.y == 0, &src, &dst);
  const int64_t mine = at.c * p.S + at.j * kQ;
  float A[kQ], h[kQ] = {};
#pragma unroll
  for (int k = 0; k < kQ; ++k) A[k] = k < at.n ? p.A[mine + k] * kLog2e : 0.f;
  if (src) load_states(src + mine, at.n, p.quad_states, h);
  float *chunk = p.chunks ? p.chunks + (b / kSsmChunk + i) * p.C * p.S + mine : nullptr;
  for (int64_t row = b; row < e; row += kSsmTile) {
    const int rows = (int)min((int64_t)kSsmTile, e - row);
    float xs[PAIRS];
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
      const int t = (k * kSsmThreads + threadIdx.x) / CH, c = threadIdx.x % CH;
      float v = 0.f;
      xs[k] = 0.f;
      if (t < rows && c < at.cn) {
        v = load_step<T>(p, row + t, at.c0 + c);
        if (p.softplus) v = softplus(v);
        xs[k] = to_f32(static_cast<const T *>(p.x)[(row + t) * p.x_st + at.c0 + c]);
      }
      steps[t][c] = make_float2(v, v * xs[k]);
    }
    load_vectors<T, SP>(p, at.g, row, rows, Bs, Cs);
    __syncthreads();
    for (int t = 0; t < rows; ++t) {
      if (chunk && t % kSsmChunk == 0) {
        store_states(chunk, at.n, p.quad_states, h);
        chunk += p.C * p.S;
      }
      const float2 d = steps[t][at.ch];
      const float4 Bt = *reinterpret_cast<const float4 *>(&Bs[t][at.j * kQ]), Ct = *reinterpret_cast<const float4 *>(&Cs[t][at.j * kQ]);
      const float bt[kQ] = {Bt.x, Bt.y, Bt.z, Bt.w}, ct[kQ] = {Ct.x, Ct.y, Ct.z, Ct.w};
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < kQ; ++k)
        if (k < at.n) {
          h[k] = fmaf(ex2(d.x * A[k]), h[k], d.y * bt[k]);
          y = fmaf(ct[k], h[k], y);
        }
      sum_scatter<1, L, 1>(&y, at.j);
      if (at.j == 0) ys[t][at.ch] = y;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
      const int t = (k * kSsmThreads + threadIdx.x) / CH, c = threadIdx.x % CH;
      if (t < rows && c < at.cn) {
        float y = ys[t][c];
        if (p.D) y = fmaf(p.D[at.c0 + c], xs[k], y);
        if (p.z) {
          const float z = to_f32(static_cast<const T *>(p.z)[(row + t) * p.z_st + at.c0 + c]);
          y *= z * sigmoid_fast(z);
        }
        static_cast<T *>(p.y)[(row + t) * p.C + at.c0 + c] = from_f32<T>(y);
      }
    }
    __syncthreads();
  }
  if (dst) store_states(dst + mine, at.n, p.quad_states, h);
}

// One token per sequence: the states are read and written once.
template <typename T, int L>
__global__ void __launch_bounds__(kSsmThreads) gdp_ssm_step_kernel(const SsmProblem p) {
  const SsmPlace<L> at(p, blockIdx.y);
  const int64_t i = blockIdx.x;
  const float *src;
  float *dst;
  state_of<float>(p.s, i, p.C * p.S, p.p.status, threadIdx.x == 0 && blockIdx.y == 0, &src, &dst);
  const bool real = at.ch < at.cn;
  const int64_t mine = at.c * p.S + at.j * kQ;
  float h[kQ] = {}, v = 0.f, x = 0.f, y = 0.f;
  if (src) load_states(src + mine, at.n, p.quad_states, h);
  if (real) {
    v = load_step<T>(p, i, at.c);
    if (p.softplus) v = softplus(v);
    x = to_f32(static_cast<const T *>(p.x)[i * p.x_st + at.c]);
  }
  const T *B = static_cast<const T *>(p.B) + i * p.B_st + at.g * p.B_sg + at.j * kQ,
          *Cm = static_cast<const T *>(p.Cm) + i * p.C_st + at.g * p.C_sg + at.j * kQ;
#pragma unroll
  for (int k = 0; k < kQ; ++k)
    if (k < at.n) {
      h[k] = fmaf(ex2(v * (p.A[mine + k] * kLog2e)), h[k], v * x * to_f32(B[k]));
      y = fmaf(to_f32(Cm[k]), h[k], y);
    }
  sum_scatter<1, L, 1>(&y, at.j);
  if (dst) store_states(dst + mine, at.n, p.quad_states, h);
  if (real && at.j == 0) {
    if (p.D) y = fmaf(p.D[at.c], x, y);
    if (p.z) {
      const float z = to_f32(static_cast<const T *>(p.z)[i * p.z_st + at.c]);
      y *= z * sigmoid_fast(z);
    }
    static_cast<T *>(p.y)[i * p.C + at.c] = from_f32<T>(y);
  }
}

// Backward: chunk by chunk from a sequence's end.  The states of a chunk's sixteen tokens are formed again from the
// entering one and stay in registers, with their decays, until the same loop has gone back over them.
template <typename T, int L>
__global__ void __launch_bounds__(kSsmThreads) gdp_ssm_bwd_kernel(const SsmProblem p) {
  using Place = SsmPlace<L>;
  constexpr int CH = Place::CH, SP = Place::SP, K = kSsmChunk, PAIRS = K * CH / kSsmThreads, R = 32 / L, W = kSsmThreads / 32;
  constexpr int kept = 2 * kQ > R ? 2 * kQ / R : 1;  // sums over the warp's channels that a lane ends up with
  __shared__ float2 steps[K][CH];  // e, e x
  __shared__ float grow[K][CH];    // dy
  __shared__ __align__(16) float Bs[K][SP], Cs[K][SP];
  __shared__ float us[K][CH], vs[K][CH], ys[K][CH];
  __shared__ float sums[W][K][2 * SP];
  const Place at(p, blockIdx.y);
  const int warp = threadIdx.x / 32, rank = threadIdx.x % 32 / L;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_packed(p.p);
  if (blockIdx.x == p.workers) {
    zero_tail<T>(p, static_cast<T *>(p.dx), at.c0, at.cn);
    zero_tail<T>(p, static_cast<T *>(p.dz), at.c0, at.cn);
    if (p.dt_f32) zero_tail<float>(p, static_cast<float *>(p.ddt), at.c0, at.cn);
    else zero_tail<T>(p, static_cast<T *>(p.ddt), at.c0, at.cn);
    return;
  }
  const int64_t mine = at.c * p.S + at.j * kQ;
  float A[kQ], dA[kQ] = {};
#pragma unroll
  for (int k = 0; k < kQ; ++k) A[k] = k < at.n ? p.A[mine + k] : 0.f;
  float dD = 0.f, dbias = 0.f;  // of channel threadIdx.x % CH, the thread's rows
  for (int64_t i = blockIdx.x; i < p.p.N; i += p.workers) {
    int64_t b, e;
    seq_rows(p.p, i, &b, &e);
    const int64_t chunks = (e - b + K - 1) / K;
    float back[kQ] = {};  // exp(e A) H of the token after
    if (p.dfin) load_states(p.dfin + i * p.C * p.S + mine, at.n, p.quad_states, back);
    for (int64_t q = chunks - 1; q >= 0; --q) {
      const int64_t row = b + q * K;
      const int rows = (int)min((int64_t)K, e - row);
      float xk[PAIRS], ek[PAIRS], slope[PAIRS], dk[PAIRS];
#pragma unroll
      for (int k = 0; k < PAIRS; ++k) {
        const int t = (k * kSsmThreads + threadIdx.x) / CH, c = threadIdx.x % CH;
        float v = 0.f, x = 0.f, d = 0.f;
        slope[k] = 1.f;
        dk[k] = 0.f;
        if (t < rows && c < at.cn) {
          const int64_t col = at.c0 + c;
          v = load_step<T>(p, row + t, col);
          if (p.softplus) {
            slope[k] = sigmoid_fast(v);
            v = softplus(v);
          }
          x = to_f32(static_cast<const T *>(p.x)[(row + t) * p.x_st + col]);
          d = dk[k] = to_f32(static_cast<const T *>(p.dy)[(row + t) * p.dy_st + col]);
          if (p.z) {
            const float z = to_f32(static_cast<const T *>(p.z)[(row + t) * p.z_st + col]);
            d *= z * sigmoid_fast(z);
          }
        }
        steps[t][c] = make_float2(v, v * x);
        grow[t][c] = d;
        xk[k] = x;
        ek[k] = v;
      }
      load_vectors<T, SP>(p, at.g, row, rows, Bs, Cs);
      float h[kQ];
      load_states(p.chunks + (b / K + i + q) * p.C * p.S + mine, at.n, p.quad_states, h);
      __syncthreads();
      float before[K][kQ], decay[K][kQ];
#pragma unroll
      for (int t = 0; t < K; ++t) {
        if (t < rows) {
          const float2 d = steps[t][at.ch];
          float y = 0.f;
#pragma unroll
          for (int k = 0; k < kQ; ++k) {
            before[t][k] = h[k];
            decay[t][k] = ex2(d.x * (A[k] * kLog2e));
            if (k < at.n) {
              h[k] = fmaf(decay[t][k], h[k], d.y * Bs[t][at.j * kQ + k]);
              y = fmaf(Cs[t][at.j * kQ + k], h[k], y);
            }
          }
          if (p.z) {
            sum_scatter<1, L, 1>(&y, at.j);
            if (at.j == 0) ys[t][at.ch] = y;
          }
        }
      }
      float dAk[kQ] = {};
#pragma unroll
      for (int t = K - 1; t >= 0; --t) {
        if (t < rows) {
          const float2 d = steps[t][at.ch];
          const float g = grow[t][at.ch];
          float u = 0.f, v = 0.f, s[2 * kQ];
#pragma unroll
          for (int k = 0; k < kQ; ++k) {
            s[k] = s[kQ + k] = 0.f;
            if (k < at.n) {
              const float H = fmaf(g, Cs[t][at.j * kQ + k], back[k]);
              s[k] = H * d.y;
              s[kQ + k] = g * (t + 1 < K && t + 1 < rows ? before[t + 1 < K ? t + 1 : t][k] : h[k]);
              u = fmaf(H, Bs[t][at.j * kQ + k], u);
              back[k] = H * decay[t][k];
              const float w = back[k] * before[t][k];
              v = fmaf(w, A[k], v);
              dAk[k] = fmaf(w, d.x, dAk[k]);
            }
          }
          sum_scatter<1, L, 1>(&u, at.j);
          sum_scatter<1, L, 1>(&v, at.j);
          if (at.j == 0) {
            us[t][at.ch] = u;
            vs[t][at.ch] = v;
          }
          sum_scatter<2 * kQ, R, L>(s, rank);
#pragma unroll
          for (int k = 0; k < kept; ++k) {
            const int which = rank * kept + k;  // state of dB, then of dC
            sums[warp][t][(which / kQ) * SP + at.j * kQ + which % kQ] = s[k];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kQ; ++k) dA[k] += dAk[k];
      __syncthreads();
      float dDk = 0.f, dbk = 0.f;
#pragma unroll
      for (int k = 0; k < PAIRS; ++k) {
        const int t = (k * kSsmThreads + threadIdx.x) / CH, c = threadIdx.x % CH;
        if (t < rows && c < at.cn) {
          const int64_t col = at.c0 + c;
          const float g = grow[t][c], u = us[t][c], D = p.D ? p.D[col] : 0.f;
          const float dt = fmaf(u, xk[k], vs[t][c]) * slope[k];
          static_cast<T *>(p.dx)[(row + t) * p.C + col] = from_f32<T>(fmaf(u, ek[k], g * D));
          if (p.dt_f32) static_cast<float *>(p.ddt)[(row + t) * p.C + col] = dt;
          else static_cast<T *>(p.ddt)[(row + t) * p.C + col] = from_f32<T>(dt);
          dDk = fmaf(g, xk[k], dDk);
          dbk += dt;
          if (p.z) {
            const float z = to_f32(static_cast<const T *>(p.z)[(row + t) * p.z_st + col]), s = sigmoid_fast(z);
            const float y = fmaf(D, xk[k], ys[t][c]);
            static_cast<T *>(p.dz)[(row + t) * p.C + col] = from_f32<T>(dk[k] * y * (s * fmaf(z, 1.f - s, 1.f)));
          }
        }
      }
      dD += dDk;
      dbias += dbk;
      for (int k = threadIdx.x; k < rows * 2 * SP; k += kSsmThreads) {
        const int t = k / (2 * SP), s = k % (2 * SP);
        float v = sums[0][t][s];
#pragma unroll
        for (int w = 1; w < W; ++w) v += sums[w][t][s];
        p.over_channels[((int64_t)blockIdx.y * p.p.T + row + t) * (2 * SP) + s] = v;
      }
      __syncthreads();
    }
    if (p.dinit) store_states(p.dinit + i * p.C * p.S + mine, at.n, p.quad_states, back);
  }
  float *out = p.over_rows + (int64_t)blockIdx.x * p.C * (p.S + 2);
#pragma unroll
  for (int k = 0; k < kQ; ++k)
    if (k < at.n) out[mine + k] = dA[k];
  // dD and ddt_bias: a channel's rows are spread over the threads that share its number
  float *share = &us[0][0], *other = &vs[0][0];
  constexpr int per = kSsmThreads / CH;
  static_assert(per <= K, "one value per thread fits");
  share[threadIdx.x] = dD;
  other[threadIdx.x] = dbias;
  __syncthreads();
  if (threadIdx.x < at.cn) {
    float a = 0.f, c = 0.f;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      a += share[k * CH + threadIdx.x];
      c += other[k * CH + threadIdx.x];
    }
    out[p.C * p.S + at.c0 + threadIdx.x] = a;
    out[p.C * (p.S + 1) + at.c0 + threadIdx.x] = c;
  }
}

// dB and dC: the sums over the CTAs that share a group's channels, in their order; padding rows are zeros.
template <typename T>
__global__ void __launch_bounds__(256) gdp_ssm_vectors_kernel(const SsmProblem p, int SP) {
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = k / (2 * SP), g = blockIdx.y;
  if (row >= p.p.T) return;
  const int s = (int)(k % (2 * SP)), state = s % SP;
  if (state >= p.S) return;
  float v = 0.f;
  if (row < cu_at(p.p, p.p.N)) {
    const float *from = p.over_channels + (g * p.tiles * p.p.T + row) * (2 * SP) + s;
#pragma unroll 4
    for (int64_t i = 0; i < p.tiles; ++i) v += from[i * p.p.T * (2 * SP)];
  }
  static_cast<T *>(s < SP ? p.dB : p.dC)[(row * p.G + g) * p.S + state] = from_f32<T>(v);
}

template <typename T>
cudaError_t launch_ssm_fwd(const SsmProblem &p, cudaStream_t stream) {
  const dim3 grid((unsigned)(p.p.N + (p.zero_pad ? 1 : 0)), (unsigned)(p.G * p.tiles));
  const int lanes = ssm_lanes(p.S);
  if (lanes == 4) gdp_ssm_fwd_kernel<T, 4><<<grid, kSsmThreads, 0, stream>>>(p);
  else if (lanes == 8) gdp_ssm_fwd_kernel<T, 8><<<grid, kSsmThreads, 0, stream>>>(p);
  else gdp_ssm_fwd_kernel<T, 16><<<grid, kSsmThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_ssm_step(const SsmProblem &p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.p.N, (unsigned)(p.G * p.tiles));
  const int lanes = ssm_lanes(p.S);
  if (lanes == 4) gdp_ssm_step_kernel<T, 4><<<grid, kSsmThreads, 0, stream>>>(p);
  else if (lanes == 8) gdp_ssm_step_kernel<T, 8><<<grid, kSsmThreads, 0, stream>>>(p);
  else gdp_ssm_step_kernel<T, 16><<<grid, kSsmThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_ssm_bwd(const SsmProblem &p, cudaStream_t stream) {
  const dim3 grid((unsigned)(p.workers + 1), (unsigned)(p.G * p.tiles));
  const int lanes = ssm_lanes(p.S), SP = lanes * kQ;
  if (lanes == 4) gdp_ssm_bwd_kernel<T, 4><<<grid, kSsmThreads, 0, stream>>>(p);
  else if (lanes == 8) gdp_ssm_bwd_kernel<T, 8><<<grid, kSsmThreads, 0, stream>>>(p);
  else gdp_ssm_bwd_kernel<T, 16><<<grid, kSsmThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.p.T > 0) gdp_ssm_vectors_kernel<T><<<dim3((unsigned)((p.p.T * 2 * SP + 255) / 256), (unsigned)p.G), 256, 0, stream>>>(p, SP);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace gdp
