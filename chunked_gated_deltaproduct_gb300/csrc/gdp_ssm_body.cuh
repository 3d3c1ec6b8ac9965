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
// would notice) is put right to first order.
__device__ __forceinline__ float2 exp_neg_abs2(float2 v) {
  const float2 a = make_float2(-fabsf(v.x), -fabsf(v.y));
  const float2 t = mul2(a, both(kLog2e));
  float2 rest = fma2(a, both(kLog2e), make_float2(-t.x, -t.y));  // what t's rounding left out
  rest = fma2(a, both((float)(1.4426950408889634074 - (double)kLog2e)), rest);
  const float2 w = make_float2(ex2(t.x), ex2(t.y));
  // (w is 0 where t is -inf and rest is no number)
  return make_float2(t.x < -126.f ? w.x : fmaf(w.x, 0.6931471806f * rest.x, w.x), t.y < -126.f ? w.y : fmaf(w.y, 0.6931471806f * rest.y, w.y));
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

// Piece r of the packed sequences: whole sequences, or pieces of p.piece tokens (piece q of sequence i is row
// cu_seqlens[i] / p.piece + i + q; the rows between are empty).
struct SsmPiece {
  int64_t i, b, e;  // sequence and rows
  int64_t chunk;    // row of its first chunk state
  bool last;        // it ends the sequence
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
    last = true;
    if (p.piece) {
      q = max((int64_t)0, r - (b / p.piece + i));
      chunk += q * (p.piece / kSsmChunk);
      b = min(b + q * p.piece, e);
      last = b + p.piece >= e;
      e = min(b + p.piece, e);
    }
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

// ---- forward: half of the CTA's warps run states, the other half feed them ----
//
// Per tile of 32 tokens the feeding warps bring the rows ahead (16-byte asynchronous copies into a ring of shared-memory
// stages), form e and e x of the next tile, and finish the outputs of the last one, while the running warps take their
// states over the present one: two channels by four states a lane, so that B and C are loaded once for both.

template <typename T>
__device__ __forceinline__ float2 load_pair(const unsigned char *raw, int i) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float2 *>(raw + 4 * i);
  else return widen<T>(*reinterpret_cast<const uint32_t *>(raw + 2 * i));
}

// The raw rows of a tile in shared memory.
template <typename T, int CH, int SP>
struct SsmStage {
  unsigned char *x, *dt, *z, *B, *C;
};
template <typename T, int CH, int SP>
__host__ __device__ constexpr int ssm_stage_bytes(int dt_size, bool gated) {
  return kSsmTile * (CH * ((int)sizeof(T) * (gated ? 2 : 1) + dt_size) + 2 * SP * (int)sizeof(T));
}
template <typename T, int L, int CPT>
constexpr int ssm_fwd_bytes(int dt_size, bool gated) {
  constexpr int CH = kSsmThreads / L, SP = L * kQ;
  return kSsmStages * ssm_stage_bytes<T, CH, SP>(dt_size, gated) + 2 * kSsmTile * (CH * 12 + ssm_skew(CPT) * 4 + SP * 8);
}

// Rows [row, row + rows) of a tensor into a stage [tile][PITCH], columns from c0 on; columns from `real` on become zeros.
template <typename T, int PITCH, int THREADS>
__device__ __forceinline__ void fill(unsigned char *to, const void *base, int64_t stride, int64_t c0, int real, int64_t row, int rows, int fast,
                                     int thread) {
  const T *from = static_cast<const T *>(base) + row * stride + c0;
  if (fast) {
    constexpr int E = 16 / sizeof(T), PER = PITCH / E, EACH = (kSsmTile * PER + THREADS - 1) / THREADS;
    static_assert(THREADS % PER == 0, "a thread keeps its columns");
    const int t0 = thread / PER, c = thread % PER * E;
    const uint32_t bytes = c < real ? 16u : 0u;
    const T *at = from + t0 * stride + (c < real ? c : 0);
    unsigned char *put = to + (t0 * PITCH + c) * sizeof(T);
#pragma unroll
    for (int k = 0; k < EACH; ++k, at += THREADS / PER * stride, put += THREADS / PER * PITCH * sizeof(T))
      if (t0 + k * (THREADS / PER) < rows) sm100::cp_async16(put, at, bytes);
  } else {
    T *at = reinterpret_cast<T *>(to);
#pragma unroll 8
    for (int i = thread; i < rows * PITCH; i += THREADS) {
      const int t = i / PITCH, c = i % PITCH;
      at[i] = c < real ? from[t * stride + c] : from_f32<T>(0.f);
    }
  }
}

template <typename T, int L, int CPT, bool FULL, bool LOCAL>
__global__ void __launch_bounds__(kSsmFeed + kSsmThreads / CPT, 3) gdp_ssm_fwd_kernel(const SsmProblem p) {
  constexpr int CH = kSsmThreads / L, SP = L * kQ, CP = CH / 2, HT = kSsmFeed, RT = kSsmThreads / CPT, YP = CH + ssm_skew(CPT);
  extern __shared__ __align__(128) unsigned char smem[];
  const int dt_size = p.dt_f32 ? 4 : (int)sizeof(T);
  const int stage_bytes = ssm_stage_bytes<T, CH, SP>(dt_size, p.z != nullptr);
  float2 *steps = reinterpret_cast<float2 *>(smem);                        // [2][tile][CH]: e, e x
  float *Bs = reinterpret_cast<float *>(steps + 2 * kSsmTile * CH);        // [2][tile][SP]
  float *Cs = Bs + 2 * kSsmTile * SP;                                      // [2][tile][SP]
  float *ys = Cs + 2 * kSsmTile * SP;                                      // [2][tile][YP]
  unsigned char *ring = reinterpret_cast<unsigned char *>(ys + 2 * kSsmTile * YP);
  const unsigned across = (unsigned)(p.G * p.tiles), tile = blockIdx.x % across;  // all channels of a piece, then the next one
  const int64_t r = blockIdx.x / across, g = tile / p.tiles, c0 = g * p.per + (tile % p.tiles) * CH;
  const int cn = (int)min((int64_t)CH, (g + 1) * p.per - c0);
  if (blockIdx.x == 0 && !LOCAL) check_packed(p.p);
  if (LOCAL) sm100::pdl_trigger();
  if (r == p.pieces) {
    if (p.piece) sm100::pdl_wait();
    zero_tail<T>(p, static_cast<T *>(p.y), c0, cn);
    return;
  }
  const SsmPiece at_rows(p, r);
  const int64_t b = at_rows.b, e = at_rows.e;
  if (p.piece && (b >= e || (LOCAL && at_rows.last))) {
    if (!LOCAL) sm100::pdl_wait();
    return;
  }
  const int tiles = (int)((e - b + kSsmTile - 1) / kSsmTile);
  const int lane = threadIdx.x % 32;
  if (threadIdx.x < RT) {
    const int j = lane % L, ch = threadIdx.x / L * CPT;  // first of CPT channels
    const int64_t mine = (c0 + ch) * p.S + j * kQ;
    const float *src = nullptr;
    float *dst = nullptr;
    if (!LOCAL) {
      state_of<float>(p.s, at_rows.i, p.C * p.S, p.p.status, threadIdx.x == 0 && tile == 0, &src, &dst);
      if (p.piece) {
        sm100::pdl_wait();  // the feeding warps read inputs only, and need not
        src = p.enter + r * p.C * p.S;
      }
      if (!at_rows.last) dst = nullptr;
    }
    int n[CPT];
    float2 A[CPT][2], h[CPT][2];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      n[k] = ch + k < cn ? max(0, min(kQ, (int)p.S - j * kQ)) : 0;
      float v[kQ] = {};
      if (src) load_states(src + mine + k * p.S, n[k], p.quad_states, v);
      h[k][0] = make_float2(v[0], v[1]);
      h[k][1] = make_float2(v[2], v[3]);
#pragma unroll
      for (int q = 0; q < kQ; ++q) v[q] = q < n[k] ? p.A[mine + k * p.S + q] * kLog2e : 0.f;
      A[k][0] = make_float2(v[0], v[1]);
      A[k][1] = make_float2(v[2], v[3]);
    }
    float *chunk = !LOCAL && p.chunks ? p.chunks + at_rows.chunk * p.C * p.S + mine : nullptr;
    float span[CPT] = {};  // sum of e over the piece
    const int states = max(0, min(kQ, (int)p.S - j * kQ));
    struct Token {
      float2 d[CPT];  // e, e x
      float4 B, C;    // the lane's part
    };
    auto load = [&](int t) {
      Token v;
      if constexpr (CPT == 2) {
        const float4 d = *reinterpret_cast<const float4 *>(steps + t * CH + ch);
        v.d[0] = make_float2(d.x, d.y);
        v.d[CPT - 1] = make_float2(d.z, d.w);
      } else {
        v.d[0] = steps[t * CH + ch];
      }
      v.B = *reinterpret_cast<const float4 *>(Bs + t * SP + j * kQ);
      if (!LOCAL) v.C = *reinterpret_cast<const float4 *>(Cs + t * SP + j * kQ);
      return v;
    };
    // One token: the states move on, y is the lane's part of the channels' readout.
    auto step = [&](const Token &in, float *y) {
      const float2 Bv[2] = {make_float2(in.B.x, in.B.y), make_float2(in.B.z, in.B.w)}, Cv[2] = {make_float2(in.C.x, in.C.y), make_float2(in.C.z, in.C.w)};
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        float2 sum;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 t = mul2(both(in.d[k].x), A[k][q]);
          float2 add = mul2(both(in.d[k].y), Bv[q]);
          if (!FULL) {  // padded states stay zero, whatever the input is
            add.x = 2 * q < states ? add.x : 0.f;
            add.y = 2 * q + 1 < states ? add.y : 0.f;
          }
          h[k][q] = fma2(make_float2(ex2(t.x), ex2(t.y)), h[k][q], add);
          if (!LOCAL) sum = q ? fma2(Cv[q], h[k][q], sum) : mul2(Cv[q], h[k][q]);
        }
        if (LOCAL) span[k] += in.d[k].x;
        else y[k] = sum.x + sum.y;
      }
    };
    // The readouts of BT tokens from t on (y: token by token, all channels): their shuffles overlap.
    constexpr int BT = kSsmChunk / CPT;
    auto readout = [&](int t, float (&y)[BT * CPT]) {
      sum_scatter<BT * CPT, L, 1>(y, j);
      constexpr int EACH = BT * CPT / L;  // sums of a lane
      const int first = j * EACH;
      float *out = ys + (t + first / CPT) * YP + ch + first % CPT;
#pragma unroll
      for (int k = 0; k < EACH; k += CPT) {
        if constexpr (CPT == 2 && EACH >= 2) *reinterpret_cast<float2 *>(out + k / CPT * YP) = make_float2(y[k], y[k + CPT - 1]);
        else out[k / CPT * YP] = y[k];
      }
    };
    auto save = [&](float *to) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float v[kQ] = {h[k][0].x, h[k][0].y, h[k][1].x, h[k][1].y};
        store_states(to + k * p.S, n[k], p.quad_states, v);
      }
    };
    __syncthreads();
    for (int k = 0; k < tiles; ++k) {
      const int rows = (int)min((int64_t)kSsmTile, e - b - (int64_t)k * kSsmTile), at = (k & 1) * kSsmTile;
      for (int t = 0; t < rows; t += kSsmChunk) {
        if (chunk) {
          save(chunk);
          chunk += p.C * p.S;
        }
        if (t + kSsmChunk <= rows) {  // four tokens at a time, the next ones' operands on their way
          Token now[4], next[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) now[u] = load(at + t + u);
#pragma unroll
          for (int w = 0; w < kSsmChunk; w += BT) {
            float y[BT * CPT];
#pragma unroll
            for (int v = 0; v < BT; v += 4) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (w + v + 4 < kSsmChunk) next[u] = load(at + t + w + v + 4 + u);
#pragma unroll
              for (int u = 0; u < 4; ++u) step(now[u], y + CPT * (v + u));
#pragma unroll
              for (int u = 0; u < 4; ++u) now[u] = next[u];
            }
            if (!LOCAL) readout(at + t + w, y);
          }
        } else {
#pragma unroll 1
          for (int v = t; v < rows; ++v) {
            float y[CPT];
            step(load(at + v), y);
            if (!LOCAL)
#pragma unroll
              for (int c = 0; c < CPT; ++c) {
                sum_scatter<1, L, 1>(y + c, j);
                if (j == 0) ys[(at + v) * YP + ch + c] = y[c];
              }
          }
        }
      }
      __syncthreads();
    }
    if (dst) save(dst + mine);
    if (LOCAL) {
      save(p.enter + r * p.C * p.S + mine);
      if (j == 0)
#pragma unroll
        for (int k = 0; k < CPT; ++k)
          if (ch + k < cn) p.spans[r * p.C + c0 + ch + k] = span[k];
    }
    return;
  }
  // ---- feeding ----
  const int thread = threadIdx.x - RT, c = thread % CP * 2;  // first of the thread's two channels
  const float bias[2] = {p.bias && c < cn ? p.bias[c0 + c] : 0.f, p.bias && c + 1 < cn ? p.bias[c0 + c + 1] : 0.f};
  const float D[2] = {p.D && c < cn ? p.D[c0 + c] : 0.f, p.D && c + 1 < cn ? p.D[c0 + c + 1] : 0.f};
  auto stage = [&](int k) {
    SsmStage<T, CH, SP> s;
    s.x = ring + (k % kSsmStages) * stage_bytes;
    s.B = s.x + kSsmTile * CH * sizeof(T);
    s.C = s.B + kSsmTile * SP * sizeof(T);
    s.dt = s.C + kSsmTile * SP * sizeof(T);
    s.z = s.dt + kSsmTile * CH * dt_size;
    return s;
  };
  auto rows_of = [&](int k) { return (int)min((int64_t)kSsmTile, e - b - (int64_t)k * kSsmTile); };
  auto bring = [&](int k) {
    if (k < tiles) {
      const int64_t row = b + (int64_t)k * kSsmTile;
      const int rows = rows_of(k);
      const SsmStage<T, CH, SP> s = stage(k);
      fill<T, CH, HT>(s.x, p.x, p.x_st, c0, cn, row, rows, p.fast_rows, thread);
      if (p.dt_f32) fill<float, CH, HT>(s.dt, p.dt, p.dt_st, c0, cn, row, rows, p.fast_rows, thread);
      else fill<T, CH, HT>(s.dt, p.dt, p.dt_st, c0, cn, row, rows, p.fast_rows, thread);
      if (!LOCAL && p.z) fill<T, CH, HT>(s.z, p.z, p.z_st, c0, cn, row, rows, p.fast_rows, thread);
      fill<T, SP, HT>(s.B, p.B, p.B_st, g * p.B_sg, (int)p.S, row, rows, p.fast_vectors, thread);
      if (!LOCAL) fill<T, SP, HT>(s.C, p.Cm, p.C_st, g * p.C_sg, (int)p.S, row, rows, p.fast_vectors, thread);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // (Rows behind the sequence's last one hold anything; what is formed of them is not used.)
  constexpr int ITEMS = kSsmTile * CP / HT, STEP = HT / CP, TOGETHER = ITEMS < 4 ? ITEMS : 4;
  auto form = [&](int k) {
    const SsmStage<T, CH, SP> s = stage(k);
    const int at = (k & 1) * kSsmTile, t0 = thread / CP;
#pragma unroll
    for (int m = 0; m < ITEMS; m += TOGETHER) {
      float2 v[TOGETHER], x[TOGETHER];
      if (p.dt_f32) {
#pragma unroll
        for (int u = 0; u < TOGETHER; ++u) v[u] = load_pair<float>(s.dt, (t0 + (m + u) * STEP) * CH + c);
      } else {
#pragma unroll
        for (int u = 0; u < TOGETHER; ++u) v[u] = load_pair<T>(s.dt, (t0 + (m + u) * STEP) * CH + c);
      }
#pragma unroll
      for (int u = 0; u < TOGETHER; ++u) x[u] = load_pair<T>(s.x, (t0 + (m + u) * STEP) * CH + c);
#pragma unroll
      for (int u = 0; u < TOGETHER; ++u) v[u] = add2(v[u], make_float2(bias[0], bias[1]));
      if (p.softplus)
#pragma unroll
        for (int u = 0; u < TOGETHER; ++u) v[u] = softplus2(v[u]);
#pragma unroll
      for (int u = 0; u < TOGETHER; ++u) {
        const float2 in = mul2(v[u], x[u]);
        *reinterpret_cast<float4 *>(steps + (at + t0 + (m + u) * STEP) * CH + c) = make_float4(v[u].x, in.x, v[u].y, in.y);
      }
    }
    constexpr int QUADS = kSsmTile * SP / kQ / HT;
    static_assert(QUADS > 0 && ITEMS > 0, "every thread has a part");
#pragma unroll
    for (int q = 0; q < QUADS; ++q) {
      const int o = (thread + q * HT) * kQ;
      const float2 b0 = load_pair<T>(s.B, o), b1 = load_pair<T>(s.B, o + 2);
      *reinterpret_cast<float4 *>(Bs + at * SP + o) = make_float4(b0.x, b0.y, b1.x, b1.y);
      if (!LOCAL) {
        const float2 d0 = load_pair<T>(s.C, o), d1 = load_pair<T>(s.C, o + 2);
        *reinterpret_cast<float4 *>(Cs + at * SP + o) = make_float4(d0.x, d0.y, d1.x, d1.y);
      }
    }
  };
  auto finish = [&](int k) {
    const SsmStage<T, CH, SP> s = stage(k);
    const int rows = rows_of(k), at = (k & 1) * kSsmTile, t0 = thread / CP;
    T *out = static_cast<T *>(p.y) + (b + (int64_t)k * kSsmTile + t0) * p.C + c0 + c;
#pragma unroll
    for (int m = 0; m < ITEMS; m += TOGETHER) {
      float2 x[TOGETHER], y[TOGETHER];
#pragma unroll
      for (int u = 0; u < TOGETHER; ++u) {
        x[u] = load_pair<T>(s.x, (t0 + (m + u) * STEP) * CH + c);
        y[u] = *reinterpret_cast<const float2 *>(ys + (at + t0 + (m + u) * STEP) * YP + c);
      }
#pragma unroll
      for (int u = 0; u < TOGETHER; ++u)
        if (p.D) y[u] = fma2(make_float2(D[0], D[1]), x[u], y[u]);
      if (p.z) {
#pragma unroll
        for (int u = 0; u < TOGETHER; ++u) x[u] = load_pair<T>(s.z, (t0 + (m + u) * STEP) * CH + c);
#pragma unroll
        for (int u = 0; u < TOGETHER; ++u) y[u] = mul2(y[u], mul2(x[u], make_float2(sigmoid_fast(x[u].x), sigmoid_fast(x[u].y))));
      }
#pragma unroll
      for (int u = 0; u < TOGETHER; ++u, out += STEP * p.C) {
        if (t0 + (m + u) * STEP >= rows) continue;
        if (p.pair_out) {
          if (c < cn) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float2 *>(out) = y[u];
            else *reinterpret_cast<uint32_t *>(out) = narrow<T>(y[u]);
          }
        } else {
          if (c < cn) out[0] = from_f32<T>(y[u].x);
          if (c + 1 < cn) out[1] = from_f32<T>(y[u].y);
        }
      }
    }
  };
  auto meet = [&](int left) {  // the feeding warps' copies but the last `left` groups have landed
    if (left) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    asm volatile("bar.sync 1, %0;" ::"n"(HT) : "memory");
  };
  bring(0);
  bring(1);
  meet(1);
  if (tiles > 0) form(0);
  __syncthreads();
  for (int k = 0; k < tiles; ++k) {
    bring(k + 2);
    if (!LOCAL && k > 0) finish(k - 1);
    meet(1);
    if (k + 1 < tiles) form(k + 1);
    __syncthreads();
  }
  if (!LOCAL && tiles > 0) finish(tiles - 1);
}

// The states entering every piece of a sequence, from those that the pieces reach from zero: S' = exp(A span) S + E.
// The product of a piece's decays may leave fp32 where no state does, so it is applied as two factors, and not to
// states that it cannot change.
__device__ __forceinline__ float carry(float S, float E, float exponent) {
  const float f = ex2(0.5f * exponent);
  return (S == 0.f || isinf(S) ? S : S * f * f) + E;
}
template <int V>
__global__ void __launch_bounds__(kSsmThreads) gdp_ssm_join_kernel(const SsmProblem p) {
  const int64_t i = blockIdx.x, at = ((int64_t)blockIdx.y * kSsmThreads + threadIdx.x) * V, per = p.C * p.S;
  sm100::pdl_trigger();
  sm100::pdl_wait();
  if (at >= per) return;
  int64_t b, e;
  seq_rows(p.p, i, &b, &e);
  const float *src;
  float *dst;
  state_of<float>(p.s, i, per, p.p.status, at == 0, &src, &dst);
  float S[V] = {}, A[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (src) S[k] = src[at + k];
    A[k] = p.A[at + k] * kLog2e;
  }
  if (b == e) {  // no piece will write the final state
    if (dst)
#pragma unroll
      for (int k = 0; k < V; ++k) dst[at + k] = S[k];
    return;
  }
  const int64_t r = b / p.piece + i, n = (e - b + p.piece - 1) / p.piece, c = at / p.S;  // (V divides S)
  float *enter = p.enter + r * per + at;
  const float *spans = p.spans + r * p.C + c;
  constexpr int AHEAD = 16;  // pieces whose loads are under way at once
  for (int64_t q = 0; q < n; q += AHEAD) {
    float E[AHEAD][V], span[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (q + u + 1 < n) {
        span[u] = spans[(q + u) * p.C];
        const Vec<float, V> v = load_vec<float, V>(enter + (q + u) * per);
#pragma unroll
        for (int k = 0; k < V; ++k) E[u][k] = v.v[k];
      }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (q + u < n) {
        store_vec<float, V>(enter + (q + u) * per, S);
        if (q + u + 1 < n)
#pragma unroll
          for (int k = 0; k < V; ++k) S[k] = carry(S[k], E[u][k], A[k] * span[u]);
      }
  }
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

template <typename T, int L, int CPT, bool FULL, bool LOCAL>
cudaError_t ssm_fwd(const SsmProblem &p, cudaStream_t stream) {
  const int bytes = ssm_fwd_bytes<T, L, CPT>(p.dt_f32 ? 4 : (int)sizeof(T), p.z != nullptr);
  constexpr int most = ssm_fwd_bytes<T, L, CPT>(4, true);
  static_assert(most <= 227 * 1024, "fits an SM");
  const auto kernel = gdp_ssm_fwd_kernel<T, L, CPT, FULL, LOCAL>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  const int64_t rows = p.pieces + (!LOCAL && p.zero_pad ? 1 : 0);
  return gdp::launch_kernel(kernel, dim3((unsigned)(rows * p.G * p.tiles)), dim3(kSsmFeed + kSsmThreads / CPT), bytes, stream, p.piece && !LOCAL, p);
}
template <typename T, int L, bool FULL>
cudaError_t ssm_fwd_by(const SsmProblem &p, cudaStream_t stream) {
  if (p.piece) {
    cudaError_t e = ssm_fwd<T, L, 2, FULL, true>(p, stream);
    if (e != cudaSuccess) return e;
    const int64_t per = p.C * p.S;
    const int64_t v = p.quad_states ? kQ : 1;
    const dim3 grid((unsigned)p.p.N, (unsigned)((per / v + kSsmThreads - 1) / kSsmThreads));
    if ((e = gdp::launch_kernel(p.quad_states ? gdp_ssm_join_kernel<kQ> : gdp_ssm_join_kernel<1>, grid, dim3(kSsmThreads), 0, stream, true, p)) != cudaSuccess)
      return e;
  }
  // A CTA alone on its SM is bound by its warps' own latencies, and twice the warps with half the channels take 16 % off
  // (8192 x 4096: 321 against 384 us); where several share an SM the work counts, and loading B and C once for two
  // channels does (8 x 4096 x 4096: 809 against 836 us).
  if (FULL && !p.piece && p.pieces * p.G * p.tiles <= p.sms) return ssm_fwd<T, L, FULL ? 1 : 2, FULL, false>(p, stream);
  return ssm_fwd<T, L, 2, FULL, false>(p, stream);
}
template <typename T>
cudaError_t launch_ssm_fwd(const SsmProblem &p, cudaStream_t stream) {
  const int lanes = ssm_lanes(p.S);
  const bool full = p.S == lanes * kQ;
  if (lanes == 4) return full ? ssm_fwd_by<T, 4, true>(p, stream) : ssm_fwd_by<T, 4, false>(p, stream);
  if (lanes == 8) return full ? ssm_fwd_by<T, 8, true>(p, stream) : ssm_fwd_by<T, 8, false>(p, stream);
  return full ? ssm_fwd_by<T, 16, true>(p, stream) : ssm_fwd_by<T, 16, false>(p, stream);
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
