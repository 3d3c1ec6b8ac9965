// gdp_ssm_parts.cuh -- what the selective state space scan's kernels share.
//
// A channel's S states belong to L lanes of one warp, four each; a CTA takes 128 / L channels of one group.
#pragma once

#include "gdp_ssm.cuh"

namespace gdp {
namespace layer {

// Floats between rows of readouts, so that those of several tokens fall on different banks.
constexpr int ssm_skew(int cpt) { return cpt == 2 ? 8 : 10; }
constexpr int kSsmStages = 4; // tiles whose rows a CTA holds: finished, run, formed and on their way
constexpr int kSsmFeed = 128;  // threads that feed
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

// e^-|v| of two values, to about 2^-22: the exponent's rounding in base 2 (up to |v| 2^-24, which decays of long memory
// would notice) is put right to first order.  (Below e^-128, nothing in fp32, the exponent stands still, so that infinite
// steps stay numbers; NaN stays NaN.)
__device__ __forceinline__ float held(float v) {
  float a;
  asm("max.NaN.f32 %0, %1, 0fC3000000;" : "=f"(a) : "f"(-fabsf(v)));
  return a;
}
__device__ __forceinline__ float2 exp_neg_abs2(float2 v) {
  const float2 a = make_float2(held(v.x), held(v.y)), t = mul2(a, both(kLog2e));
  float2 rest = fma2(a, both(kLog2e), make_float2(-t.x, -t.y));  // what t's rounding left out
  rest = fma2(a, both((float)(1.4426950408889634074 - (double)kLog2e)), rest);
  const float2 w = make_float2(ex2(t.x), ex2(t.y));
  return fma2(w, mul2(rest, both(0.6931471806f)), w);
}
// log(1 + e^v) = max(v, 0) + log(1 + w) with w = e^-|v| in (0, 1]; log(1 + w) = 2 artanh(s), s = w / (2 + w) <= 1/3, by
// its power series: what is left out is below s^17 / 17 < 2^-30, and small w keep their relative precision.
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 w = exp_neg_abs2(v), d = add2(w, both(2.f));
  const float2 s = mul2(w, make_float2(rcp(d.x), rcp(d.y))), q = mul2(s, s);
  float2 r = fma2(q, both(1.f / 15.f), both(1.f / 13.f));
  r = fma2(q, r, both(1.f / 11.f));
  r = fma2(q, r, both(1.f / 9.f));
  r = fma2(q, r, both(1.f / 7.f));
  r = fma2(q, r, both(1.f / 5.f));
  r = fma2(q, r, both(1.f / 3.f));
  r = fma2(q, r, both(1.f));
  const float2 up = make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f));
  return fma2(mul2(s, r), both(2.f), up);
}
__device__ __forceinline__ float softplus(float v) { return softplus2(make_float2(v, v)).x; }

// A of a state that there is none of: every finite step leaves its decay finite (at most 16), so that zero stays zero.
constexpr float kNoState = -0x1p-126f;
// e^(e A), the exponent in base 2 (A comes times log2 e).  The hardware's exponential is low on average, in 2^-24 of the result
// by 0.1 for exponents above -2^-8, 0.3 to 0.45 down to -1/2 and 0.8 below -1, and a state that remembers n tokens is off
// by n times that, its gradients again.  So the exponent is raised by what makes 0.15 of it: more would take the first of
// these further from zero than they were (mean errors for exponents from -2^-14, -2^-13, ... -2^-1 on: -0.11 -0.11 -0.10 -0.09
// -0.09 -0.14 -0.32 -0.44 -0.43 -0.32 -0.31 -0.29 -0.37 -0.51, each 0.15 more since; dA of 8 x 4096 x 2048 x 16: 2.1e-6
// to 1.2e-6).  Where the exponent is zero it rounds away: that decay is one.
constexpr float kRaise = 0.15f * 0x1p-24f * 1.44269504f;
__device__ __forceinline__ float decay(float e, float A) { return ex2(fmaf(e, A, kRaise)); }
__device__ __forceinline__ float2 decay2(float e, float2 A) {
  const float2 t = fma2(both(e), A, both(kRaise));
  return make_float2(ex2(t.x), ex2(t.y));
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
  __device__ __forceinline__ SsmPlace(const SsmProblem &p, int tile) {
    g = tile / p.tiles;
    c0 = g * p.per + tile % p.tiles * CH;
    cn = (int)min((int64_t)CH, (g + 1) * p.per - c0);
    ch = threadIdx.x / L;
    j = threadIdx.x % L;
    n = ch < cn ? max(0, min(kQ, (int)p.S - j * kQ)) : 0;
    c = c0 + ch;
  }
};

// A CTA's threads: the sequences by length into `order`, the longest first, ties in their own order.  `lengths`: kSsmRanked
// places that are free until it returns.
struct SsmOrder {
  unsigned short order[kSsmRanked];
  __device__ __forceinline__ void rank(const SsmProblem &p, int *lengths) {
    const int n = (int)p.p.N;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      int64_t b, e;
      seq_rows(p.p, i, &b, &e);
      lengths[i] = (int)(e - b);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int mine = lengths[i];
      int before = 0;
      for (int j = 0; j < n; ++j) before += lengths[j] > mine || (lengths[j] == mine && j < i);
      order[before] = (unsigned short)i;
    }
    __syncthreads();
  }
};

// Piece r of the packed sequences: whole sequences, or pieces of p.piece tokens (piece q of sequence i is row
// cu_seqlens[i] / p.piece + i + q; the rows between are empty).
struct SsmPiece {
  int64_t i, b, e;  // sequence and rows
  int64_t chunk;    // row of its first chunk state
  bool first, last; // it begins, it ends the sequence
  __device__ __forceinline__ SsmPiece(const SsmProblem &p, int64_t r) {
    int64_t q = 0;
    i = r;
    if (p.piece) {
      int64_t lo = 0, hi = p.p.N - 1;
      while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (cu_at(p.p, mid) / p.piece + mid <= r) lo = mid;
        else hi = mid - 1;
      }
      i = lo;
    }
    seq_rows(p.p, i, &b, &e);
    chunk = b / kSsmChunk + i;
    first = last = true;
    if (p.piece) {
      q = max((int64_t)0, r - (b / p.piece + i));
      chunk += q * (p.piece / kSsmChunk);
      first = q == 0;
      b = min(b + q * p.piece, e);
      last = b + p.piece >= e;
      e = min(b + p.piece, e);
    }
  }
};

// S' = exp(A span) S + E over a piece.  The product of its decays may leave fp32 where no state does, so it is applied as
// two factors, and not to values that it cannot change.
__device__ __forceinline__ float carry(float S, float E, float exponent) {
  const float f = ex2(0.5f * exponent);
  return (S == 0.f || isinf(S) ? S : S * f * f) + E;
}

// Zeros into rows [cu_seqlens[N], T) of a [T, C] output, the CTA's channels.
template <typename T>
__device__ __forceinline__ void zero_tail(const SsmProblem &p, T *out, int64_t c0, int cn) {
  if (!out) return;
  for (int64_t t = cu_at(p.p, p.p.N) + threadIdx.x / 32; t < p.p.T; t += blockDim.x / 32)
    for (int c = threadIdx.x % 32; c < cn; c += 32) out[t * p.C + c0 + c] = from_f32<T>(0.f);
}

template <typename T>
__device__ __forceinline__ float2 load_pair(const unsigned char *raw, int i) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float2 *>(raw + 4 * i);
  else return widen<T>(*reinterpret_cast<const uint32_t *>(raw + 2 * i));
}

// A tensor's tiles of TILE rows by PITCH columns into stages [TILE][PITCH], one after the other (forwards or, with a negative
// `tile_step`, backwards) by THREADS threads; columns from `real` on become zeros.  Fast: 16-byte asynchronous copies from a
// pointer that moves on by itself (finding the rows anew for every tile was 19 of 154 instructions a token).
template <typename T, int PITCH, int THREADS, int TILE>
struct TileFeed {
  static constexpr int E = 16 / sizeof(T), PER = PITCH / E, EACH = (TILE * PER + THREADS - 1) / THREADS, APART = THREADS / PER;
  static_assert(THREADS % PER == 0, "a thread keeps its columns");
  const T *at;     // fast: the thread's first row and columns of the coming tile; else the tile's first row and column
  int64_t stride;
  // base: the tensor's first column; row: the first tile's first row
  __device__ __forceinline__ TileFeed(const T *base, int64_t stride_, int64_t row, int real, int fast, int thread) : at(base + row * stride_), stride(stride_) {
    if (fast) at += thread / PER * stride + (thread % PER * E < real ? thread % PER * E : 0);
  }
  __device__ __forceinline__ void bring(unsigned char *to, int rows, int real, int fast, int thread, int tile_step) {
    if (fast) {
      const int t0 = thread / PER, c = thread % PER * E;
      const uint32_t bytes = c < real ? 16u : 0u;
      unsigned char *put = to + thread * 16;
#pragma unroll
      for (int k = 0; k < EACH; ++k)
        if (t0 + k * APART < rows) sm100::cp_async16(put + k * THREADS * 16, at + k * APART * stride, bytes);
    } else {
      T *put = reinterpret_cast<T *>(to);
#pragma unroll 8
      for (int i = thread; i < rows * PITCH; i += THREADS) {
        const int t = i / PITCH, c = i % PITCH;
        put[i] = c < real ? at[t * stride + c] : from_f32<T>(0.f);
      }
    }
    at += tile_step * stride;
  }
};

}  // namespace layer
}  // namespace gdp
