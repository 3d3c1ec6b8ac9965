// gdp_ssm_fwd_body.cuh -- the selective state space scan's forward kernels and one-token step, instantiated by type in
// gdp_ssm_*.cu.
#pragma once

#include "gdp_ssm_parts.cuh"

namespace gdp {
namespace layer {

// ---- forward: half of the CTA's warps run states, the other half feed them ----
//
// Per tile of 32 or 64 tokens the feeding warps bring the rows ahead (16-byte asynchronous copies into a ring of shared-memory
// stages), form e and e x of the next tile, and finish the outputs of the last one, while the running warps take their
// states over the present one: two channels by four states a lane, so that B and C are loaded once for both (or one channel,
// in twice the warps).
//
// Bound by the running warps' latency and issue slots.  Two channels a lane (several CTAs on an SM): 41 instructions a running
// warp and token for its 256 states, eight a lane, of which 16 are on packed pairs and 8 are exponentials, at 8 lanes a
// clock; 64 packed requests, 84086 x 2048 x 16 gated, bf16: 959 us at three CTAs per SM; 8 x 4096 x 2048 x 16 with the chunk
// states: 495 us.  One channel a lane (a CTA alone on its SM): 8 and 4 for half the states, in twice the warps; 65536 x 4096 x
// 16: 2209 us, 34 ns a token of 128 CTAs (its exponentials alone would take 452 us, its bytes 317).

// The raw rows of a tile in shared memory.
template <typename T, int CH, int SP>
struct SsmStage {
  unsigned char *x, *dt, *z, *B, *C;
};
template <typename T, int CH, int SP, int TILE>
__host__ __device__ constexpr int ssm_stage_bytes(int dt_size, bool gated) {
  return TILE * (CH * ((int)sizeof(T) * (gated ? 2 : 1) + dt_size) + 2 * SP * (int)sizeof(T));
}
template <typename T, int L, int CPT, int TILE>
constexpr int ssm_fwd_bytes(int dt_size, bool gated) {
  constexpr int CH = kSsmThreads / L, SP = L * kQ;
  return kSsmStages * ssm_stage_bytes<T, CH, SP, TILE>(dt_size, gated) + 2 * TILE * (CH * 12 + ssm_skew(CPT) * 4 + SP * 8);
}

template <typename T, int L, int CPT, int TILE, bool FULL, bool LOCAL>
__global__ void __launch_bounds__(kSsmFeed + kSsmThreads / CPT, CPT == 1 ? 1 : kSsmForward) gdp_ssm_fwd_kernel(const SsmProblem p) {
  constexpr int CH = kSsmThreads / L, SP = L * kQ, CP = CH / 2, HT = kSsmFeed, RT = kSsmThreads / CPT, YP = CH + ssm_skew(CPT);
  extern __shared__ __align__(128) unsigned char smem[];
  const int dt_size = p.dt_f32 ? 4 : (int)sizeof(T);
  const int stage_bytes = ssm_stage_bytes<T, CH, SP, TILE>(dt_size, p.z != nullptr);
  float2 *steps = reinterpret_cast<float2 *>(smem);                        // [2][tile][CH]: e, e x
  float *Bs = reinterpret_cast<float *>(steps + 2 * TILE * CH);        // [2][tile][SP]
  float *Cs = Bs + 2 * TILE * SP;                                      // [2][tile][SP]
  float *ys = Cs + 2 * TILE * SP;                                      // [2][tile][YP]
  unsigned char *ring = reinterpret_cast<unsigned char *>(ys + 2 * TILE * YP);
  const unsigned across = (unsigned)(p.G * p.tiles), tile = blockIdx.x % across, group = tile / (unsigned)p.tiles;  // all channels of a piece, then the next one
  const int64_t r = blockIdx.x / across, g = group, c0 = g * p.per + (tile - group * p.tiles) * CH;
  const int cn = (int)min((int64_t)CH, (g + 1) * p.per - c0);
  if (blockIdx.x == 0 && !LOCAL) check_packed(p.p);
  if (LOCAL) sm100::pdl_trigger();
  if (r == p.pieces) {
    if (p.piece) sm100::pdl_wait();
    zero_tail<T>(p, static_cast<T *>(p.y), c0, cn);
    return;
  }
  __shared__ SsmOrder by_length;
  if (!LOCAL && p.ranked) by_length.rank(p, reinterpret_cast<int *>(smem));
  const SsmPiece at_rows(p, !LOCAL && p.ranked ? by_length.order[r] : r);
  const int64_t b = at_rows.b, e = at_rows.e;
  if (p.piece && (b >= e || (LOCAL && at_rows.last))) {
    if (!LOCAL) sm100::pdl_wait();
    return;
  }
  const int tiles = (int)((e - b + TILE - 1) / TILE);
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
      for (int q = 0; q < kQ; ++q) v[q] = q < n[k] ? p.A[mine + k * p.S + q] * kLog2e : kNoState;
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
          h[k][q] = fma2(decay2(in.d[k].x, A[k][q]), h[k][q], mul2(both(in.d[k].y), Bv[q]));
          if (!FULL) {  // padded states stay zero, whatever the input and the decay are (infinite ones too)
            h[k][q].x = 2 * q < states ? h[k][q].x : 0.f;
            h[k][q].y = 2 * q + 1 < states ? h[k][q].y : 0.f;
          }
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
      const int rows = (int)min((int64_t)TILE, e - b - (int64_t)k * TILE), at = (k & 1) * TILE;
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
    s.B = s.x + TILE * CH * sizeof(T);
    s.C = s.B + TILE * SP * sizeof(T);
    s.dt = s.C + TILE * SP * sizeof(T);
    s.z = s.dt + TILE * CH * dt_size;
    return s;
  };
  auto rows_of = [&](int k) { return (int)min((int64_t)TILE, e - b - (int64_t)k * TILE); };
  TileFeed<T, CH, HT, TILE> x_feed(static_cast<const T *>(p.x) + c0, p.x_st, b, cn, p.fast_rows, thread),
      z_feed(static_cast<const T *>(p.z) + (p.z ? c0 : 0), p.z_st, p.z ? b : 0, cn, p.fast_rows && p.z, thread),
      dt_feed(static_cast<const T *>(p.dt) + (p.dt_f32 ? 0 : c0), p.dt_st, p.dt_f32 ? 0 : b, cn, p.fast_rows, thread);
  TileFeed<float, CH, HT, TILE> dt32_feed(static_cast<const float *>(p.dt) + (p.dt_f32 ? c0 : 0), p.dt_st, p.dt_f32 ? b : 0, cn, p.fast_rows, thread);
  TileFeed<T, SP, HT, TILE> B_feed(static_cast<const T *>(p.B) + g * p.B_sg, p.B_st, b, (int)p.S, p.fast_vectors, thread),
      C_feed(static_cast<const T *>(p.Cm) + g * p.C_sg, p.C_st, b, (int)p.S, p.fast_vectors, thread);
  auto bring = [&](int k) {  // tile by tile
    if (k < tiles) {
      const int rows = rows_of(k);
      const SsmStage<T, CH, SP> s = stage(k);
      x_feed.bring(s.x, rows, cn, p.fast_rows, thread, TILE);
      if (p.dt_f32) dt32_feed.bring(s.dt, rows, cn, p.fast_rows, thread, TILE);
      else dt_feed.bring(s.dt, rows, cn, p.fast_rows, thread, TILE);
      if (!LOCAL && p.z) z_feed.bring(s.z, rows, cn, p.fast_rows, thread, TILE);
      B_feed.bring(s.B, rows, (int)p.S, p.fast_vectors, thread, TILE);
      if (!LOCAL) C_feed.bring(s.C, rows, (int)p.S, p.fast_vectors, thread, TILE);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // (Rows behind the sequence's last one hold anything; what is formed of them is not used.)
  constexpr int ITEMS = TILE * CP / HT, STEP = HT / CP, TOGETHER = ITEMS < 4 ? ITEMS : 4;
  auto form = [&](int k) {
    const SsmStage<T, CH, SP> s = stage(k);
    const int at = (k & 1) * TILE, t0 = thread / CP;
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
    constexpr int QUADS = TILE * SP / kQ / HT;
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
    const int rows = rows_of(k), at = (k & 1) * TILE, t0 = thread / CP;
    T *out = static_cast<T *>(p.y) + (b + (int64_t)k * TILE + t0) * p.C + c0 + c;
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
        for (int u = 0; u < TOGETHER; ++u) y[u] = mul2(y[u], mul2(x[u], sigmoid2(x[u])));
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

// The states entering every piece of a sequence, from those that the pieces reach from zero.
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

// Four values of a vector's states, n of them exist; `quad`: they can be read together.
template <typename T>
__device__ __forceinline__ void load_quad(const T *at, int n, int quad, float (&v)[kQ]) {
  if (quad && n == kQ) {
    const Vec<T, kQ> q = load_vec<T, kQ>(at);
#pragma unroll
    for (int k = 0; k < kQ; ++k) v[k] = to_f32(q.v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kQ; ++k) v[k] = k < n ? to_f32(at[k]) : 0.f;
  }
}

// One token per sequence: the states are read and written once (64 x 4096 x 16: 33.5 MB).  U sequences per CTA: A is read
// once for them, their loads are under way together, and what a (sequence, channel) pair needs once is formed by one of
// the channel's lanes for each sequence (64 x 4096 x 16 on the device: 12.5 us with every lane for itself, one sequence).
template <typename T, int L, int U>
__global__ void __launch_bounds__(kSsmThreads) gdp_ssm_step_kernel(const SsmProblem p) {
  const SsmPlace<L> at(p, blockIdx.y);
  const bool real = at.ch < at.cn;
  const int64_t mine = at.c * p.S + at.j * kQ, first = (int64_t)blockIdx.x * U, per = p.C * p.S;
  const int own = at.j % U;  // the lane's sequence
  const int64_t i = first + own;
  int64_t slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) slot[u] = p.s.cache && first + u < p.p.N ? p.s.slots[first + u] : 0;
  float A[kQ], h[U][kQ], B[U][kQ], Cm[U][kQ], v = 0.f, x = 0.f, z = 0.f;
  load_quad(p.A + mine, at.n, p.quad_vectors, A);
  if (real && i < p.p.N) {
    v = load_step<T>(p, i, at.c);
    x = to_f32(static_cast<const T *>(p.x)[i * p.x_st + at.c]);
    if (p.z) z = to_f32(static_cast<const T *>(p.z)[i * p.z_st + at.c]);
  }
  const T *B_at = static_cast<const T *>(p.B) + first * p.B_st + at.g * p.B_sg + at.j * kQ,
          *C_at = static_cast<const T *>(p.Cm) + first * p.C_st + at.g * p.C_sg + at.j * kQ;
  float *dst[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool exists = first + u < p.p.N;
    load_quad(B_at, exists ? at.n : 0, p.quad_vectors, B[u]);
    load_quad(C_at, exists ? at.n : 0, p.quad_vectors, Cm[u]);
    if (first + u + 1 < p.p.N) B_at += p.B_st, C_at += p.C_st;
    const float *src = nullptr;
    dst[u] = nullptr;
    if (p.s.cache) {
      const bool good = exists && slot[u] >= 0 && slot[u] < p.s.num_slots;
      if (exists && !good && slot[u] != -1 && threadIdx.x == 0 && blockIdx.y == 0) set_status(p.p.status, GDP_DEV_ERR_SLOT);
      if (good) src = dst[u] = static_cast<float *>(p.s.cache) + slot[u] * per + mine;
    } else if (exists) {
      if (p.s.init) src = static_cast<const float *>(p.s.init) + (first + u) * per + mine;
      if (p.s.fin) dst[u] = static_cast<float *>(p.s.fin) + (first + u) * per + mine;
    }
#pragma unroll
    for (int k = 0; k < kQ; ++k) h[u][k] = 0.f;
    if (src) load_states(src, at.n, p.quad_states, h[u]);
  }
  if (p.softplus) v = softplus(v);
  const float in = v * x;
#pragma unroll
  for (int k = 0; k < kQ; ++k) A[k] *= kLog2e;
  float y[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float e = U > 1 ? __shfl_sync(0xffffffffu, v, u, L) : v, ex = U > 1 ? __shfl_sync(0xffffffffu, in, u, L) : in;
    y[u] = 0.f;
#pragma unroll
    for (int k = 0; k < kQ; ++k)
      if (k < at.n) {
        h[u][k] = fmaf(decay(e, A[k]), h[u][k], ex * B[u][k]);
        y[u] = fmaf(Cm[u][k], h[u][k], y[u]);
      }
    if (dst[u]) store_states(dst[u], at.n, p.quad_states, h[u]);
  }
  // sequence u's readout to the channel's lane u
  float mine_y = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int k = L / 2; k > 0; k /= 2) y[u] += __shfl_xor_sync(0xffffffffu, y[u], k);
    if (own == u) mine_y = y[u];
  }
  if (real && at.j < U && i < p.p.N) {
    if (p.D) mine_y = fmaf(p.D[at.c], x, mine_y);
    if (p.z) mine_y *= z * sigmoid_fast(z);
    static_cast<T *>(p.y)[i * p.C + at.c] = from_f32<T>(mine_y);
  }
}

template <typename T, int L, int CPT, bool FULL, bool LOCAL>
cudaError_t ssm_fwd(const SsmProblem &p, cudaStream_t stream) {
  // tokens of a tile: a CTA alone on its SM takes 64 where they fit (8192 x 4096: 282 us, 32: 316), the others 32 (8 x 4096 x
  // 4096: 776 us; 64 leave room for two CTAs only, 1280; 16 meet twice as often, 923 with three CTAs, 933 with four)
  constexpr int TILE = CPT == 1 && ssm_fwd_bytes<T, L, CPT, 64>(4, true) <= 220 * 1024 ? 64 : 32;
  const int bytes = ssm_fwd_bytes<T, L, CPT, TILE>(p.dt_f32 ? 4 : (int)sizeof(T), p.z != nullptr);
  constexpr int most = ssm_fwd_bytes<T, L, CPT, TILE>(4, true);
  static_assert(most <= 227 * 1024, "fits an SM");
  const auto kernel = gdp_ssm_fwd_kernel<T, L, CPT, TILE, FULL, LOCAL>;
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
  // (8192 x 4096, both with 32 tokens a tile: 321 against 384 us; with 64 tokens 282); where several share an SM the work
  // counts, and loading B and C once for two channels does (8 x 4096 x 4096: 809 against 836 us).
  if (FULL && !p.piece && p.pieces * p.G * (int64_t)p.tiles <= p.sms) return ssm_fwd<T, L, FULL ? 1 : 2, FULL, false>(p, stream);
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
template <typename T, int L>
cudaError_t ssm_step(const SsmProblem &p, cudaStream_t stream) {
  // two sequences a CTA where there are plenty (64 x 4096 x 16: 10.4 us, one 12.8, four 12.3), one for latency
  const int64_t tiles = p.G * p.tiles;
  if (p.p.N * tiles >= 16 * p.sms) gdp_ssm_step_kernel<T, L, 2><<<dim3((unsigned)((p.p.N + 1) / 2), (unsigned)tiles), kSsmThreads, 0, stream>>>(p);
  else gdp_ssm_step_kernel<T, L, 1><<<dim3((unsigned)p.p.N, (unsigned)tiles), kSsmThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_ssm_step(const SsmProblem &p, cudaStream_t stream) {
  const int lanes = ssm_lanes(p.S);
  return lanes == 4 ? ssm_step<T, 4>(p, stream) : lanes == 8 ? ssm_step<T, 8>(p, stream) : ssm_step<T, 16>(p, stream);
}

}  // namespace layer
}  // namespace gdp
