// gdp_ssm_bwd_body.cuh -- the selective state space scan's backward kernels, instantiated by type in gdp_ssm_bwd_*.cu.
#pragma once

#include "gdp_ssm_parts.cuh"

namespace gdp {
namespace layer {

// Chunk by chunk from a piece's end.  As in the forward pass, feeding warps bring rows (and the states entering the
// chunks), form e, e x and dy, and finish gradients, while running warps hold two channels by four states a lane.  The
// states before a chunk's tokens are formed again from the entering one: once through for those before every second
// token, then two tokens at a time into registers, with their decays, which the same two going back use (four: 214 registers
// or spills).  Sums over a channel's lanes and over the CTA's channels are the feeding warps': the running ones, whose chain
// of dependent steps is what takes the time, leave their parts in shared memory, eight tokens at a time (shuffles in the
// running warps instead: training step of 8 x 4096 x 2048: 3.17 against 2.54 ms).
//
// Bound as the forward pass is, by few warps with dependent work (430 instructions a token of 32 channels, issue slots 36 %
// busy): 8 x 4096 x 2048 x 16 bf16 in 1894 us, dB and dC's parts added up in 52 more, dA's, dD's and ddt_bias's in 13.  Two CTAs
// on an SM are what its shared memory is cut to: one takes 1.6 times as long (16384 x 2048 x 16, gated, bf16 with fp32 dt: 1771
// us by one, 1046 by two; fp32 without a gate 1497 and 886; gated fp32 of 16 states is by one, 1707 us).

template <typename T, int L>
struct SsmBack {
  static constexpr int CH = kSsmThreads / L, SP = L * kQ, K = kSsmChunk, HALF = K / 2, RT = kSsmThreads / 2;
  static constexpr int STAGES = 3;  // chunks whose rows a CTA holds: finished or on their way, run, formed
  static constexpr int BLK = 2;     // tokens there and back in registers
  __host__ __device__ static constexpr int stage(int dt_size, bool gated) {
    return K * CH * ((int)sizeof(T) * (gated ? 3 : 2) + dt_size) + 2 * K * SP * (int)sizeof(T) + CH * SP * 4;
  }
  static constexpr bool WIDEN = sizeof(T) == 2;  // B and C have to be widened
  // two chunks of e and e x, dy, B and C; two halves of the running threads' parts; their states before every BLKth token but the
  // chunk's first, their sums for dA
  static constexpr int formed = K * CH * 12 + (WIDEN ? 2 * K * SP * 4 : 0), starts = K / BLK * RT * 8 * 4;
  __host__ __device__ static constexpr int parts(bool gated) { return HALF * RT * (8 + 2 * (gated ? 3 : 2)) * 4; }
  __host__ __device__ static constexpr int bytes(int dt_size, bool gated) {
    return STAGES * stage(dt_size, gated) + 2 * (formed + parts(gated)) + starts;
  }
};

template <typename T, int L, bool FULL, bool LOCAL>
__global__ void __launch_bounds__(kSsmFeed + kSsmThreads / 2, kSsmBackward) gdp_ssm_bwd_kernel(const SsmProblem p) {
  using Back = SsmBack<T, L>;
  constexpr int CH = Back::CH, SP = Back::SP, K = Back::K, HALF = Back::HALF, CP = CH / 2, HT = kSsmFeed, RT = Back::RT, BLK = Back::BLK;
  constexpr float kLn2 = 0.69314718055994531f;
  extern __shared__ __align__(128) unsigned char smem[];
  const int dt_size = p.dt_f32 ? 4 : (int)sizeof(T), stage_bytes = Back::stage(dt_size, p.z != nullptr);
  float2 *steps = reinterpret_cast<float2 *>(smem);            // [2][K][CH]: e, e x
  float *gs = reinterpret_cast<float *>(steps + 2 * K * CH);   // [2][K][CH]: dy
  float *Bs = gs + 2 * K * CH, *Cs = Bs + (Back::WIDEN ? 2 * K * SP : 0);  // [2][K][SP]
  // Parts of half a chunk: of dB and dC [2][HALF][2][RT], of u, v and y [2][HALF][kinds][L][CP].
  const int kinds = p.z ? 3 : 2;
  float4 *sums = reinterpret_cast<float4 *>(Cs + (Back::WIDEN ? 2 * K * SP : 0));
  float2 *parts = reinterpret_cast<float2 *>(sums + 2 * HALF * 2 * RT);
  float4 *starts = reinterpret_cast<float4 *>(parts + 2 * HALF * kinds * RT);  // [K / BLK - 1][2][RT]
  float4 *totals = starts + (K / BLK - 1) * 2 * RT;  // [2][RT]
  unsigned char *ring = reinterpret_cast<unsigned char *>(totals + 2 * RT);
  // (pairs of channels change places by lane, so that half a warp's parts fall on all banks)
  auto part_of = [&](int t, int kind, int j, int pair) {
    return ((t * kinds + kind) * L + j) * CP + (pair ^ (j / (L / 4) * (CP / 4)));
  };
  struct Stage {
    unsigned char *x, *dt, *dy, *z, *B, *C;
    float *h;  // [CH][S]
  };
  auto stage = [&](int k) {
    Stage s;
    s.x = ring + (k % Back::STAGES) * stage_bytes;
    s.dy = s.x + K * CH * sizeof(T);
    s.B = s.dy + K * CH * sizeof(T);
    s.C = s.B + K * SP * sizeof(T);
    s.h = reinterpret_cast<float *>(s.C + K * SP * sizeof(T));
    s.dt = reinterpret_cast<unsigned char *>(s.h + CH * SP);
    s.z = s.dt + K * CH * dt_size;
    return s;
  };
  const unsigned across = (unsigned)(p.G * p.tiles), tile = blockIdx.x % across, group = tile / (unsigned)p.tiles;
  const int64_t worker = blockIdx.x / across, g = group, c0 = g * p.per + (tile - group * p.tiles) * CH;
  const int cn = (int)min((int64_t)CH, (g + 1) * p.per - c0);
  if (blockIdx.x == 0 && !LOCAL) check_packed(p.p);
  if (LOCAL) sm100::pdl_trigger();
  if (worker == p.workers) {
    zero_tail<T>(p, static_cast<T *>(p.dx), c0, cn);
    zero_tail<T>(p, static_cast<T *>(p.dz), c0, cn);
    if (p.dt_f32) zero_tail<float>(p, static_cast<float *>(p.ddt), c0, cn);
    else zero_tail<T>(p, static_cast<T *>(p.ddt), c0, cn);
    if (p.piece) sm100::pdl_wait();
    return;
  }
  __shared__ SsmOrder by_length;
  if (!LOCAL && p.ranked) by_length.rank(p, reinterpret_cast<int *>(smem));
  auto row_of = [&](int64_t r) { return !LOCAL && p.ranked ? (int64_t)by_length.order[r] : r; };
  const bool running = threadIdx.x < RT;
  float *out = p.over_rows + worker * ssm_sum_cols(p.C, p.S);
  if (running) {
    const int j = threadIdx.x % L, ch = threadIdx.x / L * 2;
    const int64_t mine = (c0 + ch) * p.S + j * kQ;
    const int states = max(0, min(kQ, (int)p.S - j * kQ));
    int n[2];
    float2 A[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      n[k] = ch + k < cn ? states : 0;
      float v[kQ];
#pragma unroll
      for (int q = 0; q < kQ; ++q) v[q] = q < n[k] ? p.A[mine + k * p.S + q] * kLog2e : kNoState;
      A[k][0] = make_float2(v[0], v[1]);
      A[k][1] = make_float2(v[2], v[3]);
      totals[k * RT + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // padded states stay zero, whatever the inputs and the decays are, and so do their gradients (kNoState)
    auto real = [&](float2 v, int q) { return FULL ? v : make_float2(2 * q < states ? v.x : 0.f, 2 * q + 1 < states ? v.y : 0.f); };
    auto pairs = [](float4 v, float2 (&o)[2]) {
      o[0] = make_float2(v.x, v.y);
      o[1] = make_float2(v.z, v.w);
    };
    auto save = [&](float *to, const float2 (&v)[2][2]) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float o[kQ] = {v[k][0].x, v[k][0].y, v[k][1].x, v[k][1].y};
        store_states(to + k * p.S, n[k], p.quad_states, o);
      }
    };
    if (p.piece && !LOCAL) sm100::pdl_wait();
    for (int64_t r = worker; r < p.pieces; r += p.workers) {
      const SsmPiece at_rows(p, row_of(r));
      if (p.piece && (at_rows.b >= at_rows.e || (LOCAL && at_rows.first))) continue;
      const int chunks = (int)((at_rows.e - at_rows.b + K - 1) / K);
      float2 back[2][2];  // exp(e A) H of the token after
      {
        const float *from = LOCAL ? nullptr : p.piece ? p.enter + r * p.C * p.S : p.dfin ? p.dfin + at_rows.i * p.C * p.S : nullptr;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[kQ] = {};
          if (from) load_states(from + mine + k * p.S, n[k], p.quad_states, v);
          back[k][0] = make_float2(v[0], v[1]);
          back[k][1] = make_float2(v[2], v[3]);
        }
      }
      float span[2] = {};
      __syncthreads();
      for (int k = 0; k < chunks; ++k) {
        const int at = (k & 1) * K, rows = k == 0 ? (int)(at_rows.e - at_rows.b) - (chunks - 1) * K : K;
        const float *B_at = Back::WIDEN ? Bs + at * SP + j * kQ : reinterpret_cast<const float *>(stage(k).B) + j * kQ;
        const float *C_at = Back::WIDEN ? Cs + at * SP + j * kQ : reinterpret_cast<const float *>(stage(k).C) + j * kQ;
        if constexpr (LOCAL) {
#pragma unroll 4
          for (int t = rows - 1; t >= 0; --t) {
            const float4 d = *reinterpret_cast<const float4 *>(steps + (at + t) * CH + ch);
            const float2 gd = *reinterpret_cast<const float2 *>(gs + (at + t) * CH + ch);
            float2 Cv[2];
            pairs(*reinterpret_cast<const float4 *>(C_at + t * SP), Cv);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float e = c ? d.z : d.x;
              span[c] += e;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                back[c][q] = real(mul2(decay2(e, A[c][q]), fma2(both(c ? gd.y : gd.x), Cv[q], back[c][q])), q);
              }
            }
          }
        } else {
          float2 h[2][2], dA[2][2] = {};  // (a chunk's part: sums over many tokens run in two steps)
          const float *from = stage(k).h + ch * p.S + j * kQ;
          auto entering = [&] {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float v[kQ];
              load_states(from + c * p.S, n[c], FULL, v);
              h[c][0] = make_float2(v[0], v[1]);
              h[c][1] = make_float2(v[2], v[3]);
            }
          };
          entering();
          // h of the token at t from the one before; `decay` its factor
          auto forth = [&](int t, float2 (&decay)[2][2]) {
            const float4 d = *reinterpret_cast<const float4 *>(steps + (at + t) * CH + ch);
            float2 Bv[2];
            pairs(*reinterpret_cast<const float4 *>(B_at + t * SP), Bv);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                decay[c][q] = decay2(c ? d.z : d.x, A[c][q]);
                h[c][q] = real(fma2(decay[c][q], h[c][q], mul2(both(c ? d.w : d.y), Bv[q])), q);
              }
          };
          auto copy = [](float2 (&to)[2][2], const float2 (&from)[2][2]) {
#pragma unroll
            for (int c = 0; c < 2; ++c) to[c][0] = from[c][0], to[c][1] = from[c][1];
          };
          auto keep = [&](int q) {
#pragma unroll
            for (int c = 0; c < 2; ++c) starts[((q - 1) * 2 + c) * RT + threadIdx.x] = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
          };
          float2 unused[2][2];
#pragma unroll 1
          for (int q = 1; BLK * q < rows; ++q) {
#pragma unroll
            for (int u = 0; u < BLK; ++u) forth(BLK * (q - 1) + u, unused);
            keep(q);
          }
          struct Token {
            float4 d, B, C;  // e, e x of both channels; the lane's part
            float2 g;        // dy of both
          };
          auto load = [&](int t) {
            return Token{*reinterpret_cast<const float4 *>(steps + (at + t) * CH + ch), *reinterpret_cast<const float4 *>(B_at + t * SP),
                         *reinterpret_cast<const float4 *>(C_at + t * SP), *reinterpret_cast<const float2 *>(gs + (at + t) * CH + ch)};
          };
          // BLK tokens from t on (m of them exist), there and back
          auto some = [&](int t, int m, auto whole) {
            constexpr bool ALL = decltype(whole)::value;
            float2 before[BLK][2][2], decay[BLK][2][2];
#pragma unroll
            for (int w = 0; w < BLK; ++w) {
              if (!ALL && w >= m) break;
              copy(before[w], h);
              forth(t + w, decay[w]);
            }
            if (p.z) {
#pragma unroll
              for (int w = 0; w < BLK; ++w) {
                if (!ALL && w >= m) break;
                float2 Cv[2];
                float y[2];
                pairs(*reinterpret_cast<const float4 *>(C_at + (t + w) * SP), Cv);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const bool end = ALL ? w + 1 == BLK : w + 1 >= m;  // (h: after the last of them)
                  const float2 h0 = end ? h[c][0] : before[w + 1 < BLK ? w + 1 : w][c][0], h1 = end ? h[c][1] : before[w + 1 < BLK ? w + 1 : w][c][1];
                  const float2 sum = fma2(Cv[1], h1, mul2(Cv[0], h0));
                  y[c] = sum.x + sum.y;
                }
                parts[part_of(t + w, 2, j, ch / 2)] = make_float2(y[0], y[1]);
              }
            }
            Token in = load(t + (ALL ? BLK : m) - 1);
#pragma unroll
            for (int w = BLK - 1; w >= 0; --w) {
              if (!ALL && w >= m) continue;
              Token next;
              if (w > 0) next = load(t + w - 1);
              float2 Bv[2], Cv[2], sB[2], sC[2];
              float u[2], v[2];
              pairs(in.B, Bv);
              pairs(in.C, Cv);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float2 gg = both(c ? in.g.y : in.g.x), ee = both(c ? in.d.z : in.d.x), ex = both(c ? in.d.w : in.d.y);
                float2 uu, vv;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const float2 H = real(fma2(gg, Cv[q], back[c][q]), q);
                  sB[q] = c ? fma2(H, ex, sB[q]) : mul2(H, ex);
                  sC[q] = c ? fma2(gg, h[c][q], sC[q]) : mul2(gg, h[c][q]);
                  uu = q ? fma2(H, Bv[q], uu) : mul2(H, Bv[q]);
                  back[c][q] = mul2(H, decay[w][c][q]);
                  const float2 x = mul2(back[c][q], before[w][c][q]);
                  vv = q ? fma2(x, A[c][q], vv) : mul2(x, A[c][q]);
                  dA[c][q] = fma2(x, ee, dA[c][q]);
                }
                u[c] = uu.x + uu.y;
                v[c] = vv.x + vv.y;
              }
              float4 *to = sums + (t + w) * 2 * RT + threadIdx.x;
              to[0] = make_float4(sB[0].x, sB[0].y, sB[1].x, sB[1].y);
              to[RT] = make_float4(sC[0].x, sC[0].y, sC[1].x, sC[1].y);
              parts[part_of(t + w, 0, j, ch / 2)] = make_float2(u[0], u[1]);
              parts[part_of(t + w, 1, j, ch / 2)] = make_float2(v[0], v[1]);
              copy(h, before[w]);
              if (w > 0) in = next;
            }
          };
          int q = (rows - 1) / BLK;
#pragma unroll 1
          for (int half = 1; half >= 0; --half) {
            auto block = [&](int q, auto whole) {
              if (q == 0) {
                entering();
              } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) pairs(starts[((q - 1) * 2 + c) * RT + threadIdx.x], h[c]);
              }
              some(BLK * q, min(BLK, rows - BLK * q), whole);
            };
            if (rows == K) {
#pragma unroll
              for (int n = HALF / BLK - 1; n >= 0; --n) block(half * (HALF / BLK) + n, std::true_type{});
            } else {
#pragma unroll 1
              for (; q >= half * (HALF / BLK); --q) block(q, std::false_type{});
            }
            if (half == 0)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float4 &sum = totals[c * RT + threadIdx.x];
                sum = make_float4(sum.x + dA[c][0].x, sum.y + dA[c][0].y, sum.z + dA[c][1].x, sum.w + dA[c][1].y);
              }
            __syncthreads();
          }
        }
        if (LOCAL) {
          __syncthreads();
          __syncthreads();
        }
      }
      if (LOCAL) {
        save(p.enter + r * p.C * p.S + mine, back);
        if (j == 0)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (ch + k < cn) p.spans[r * p.C + c0 + ch + k] = span[k];
      } else if (p.dinit && at_rows.first) {
        save(p.dinit + at_rows.i * p.C * p.S + mine, back);
      }
    }
    if (!LOCAL) {
      float2 dA[2][2];
#pragma unroll
      for (int c = 0; c < 2; ++c) pairs(totals[c * RT + threadIdx.x], dA[c]);
      save(out + mine, dA);
    }
    return;
  }
  // ---- feeding ----
  const int thread = threadIdx.x - RT, c = thread % CP * 2, t0 = thread / CP;  // first of the thread's two channels, its first token
  constexpr int STEP = HT / CP, ITEMS = (K + STEP - 1) / STEP;
  const float bias[2] = {p.bias && c < cn ? p.bias[c0 + c] : 0.f, p.bias && c + 1 < cn ? p.bias[c0 + c + 1] : 0.f};
  const float2 D = make_float2(p.D && c < cn ? p.D[c0 + c] : 0.f, p.D && c + 1 < cn ? p.D[c0 + c + 1] : 0.f);
  // sums over the worker's rows, in two steps: over kSums chunks' and then these (their roundings grow with the shorter of the two)
  constexpr int kSums = 16;
  float2 dD = make_float2(0.f, 0.f), dbias = make_float2(0.f, 0.f), total_D = dD, total_bias = dD;
  auto add_up = [&] {
    total_D = add2(total_D, dD);
    total_bias = add2(total_bias, dbias);
    dD = dbias = make_float2(0.f, 0.f);
  };
  for (int64_t r = worker; r < p.pieces; r += p.workers) {
    const SsmPiece at_rows(p, row_of(r));
    if (p.piece && (at_rows.b >= at_rows.e || (LOCAL && at_rows.first))) continue;
    const int chunks = (int)((at_rows.e - at_rows.b + K - 1) / K);
    // step k goes over chunk chunks - 1 - k
    auto first_row = [&](int k) { return at_rows.b + (int64_t)(chunks - 1 - k) * K; };
    auto rows_of = [&](int k) { return k == 0 ? (int)(at_rows.e - at_rows.b) - (chunks - 1) * K : K; };
    const int64_t last_row = chunks > 0 ? first_row(0) : 0;
    TileFeed<T, CH, HT, K> x_feed(static_cast<const T *>(p.x) + c0, p.x_st, last_row, cn, p.fast_rows, thread),
        dy_feed(static_cast<const T *>(p.dy) + c0, p.dy_st, last_row, cn, p.fast_rows, thread),
        z_feed(static_cast<const T *>(p.z) + (p.z ? c0 : 0), p.z_st, p.z ? last_row : 0, cn, p.fast_rows && p.z, thread),
        dt_feed(static_cast<const T *>(p.dt) + (p.dt_f32 ? 0 : c0), p.dt_st, p.dt_f32 ? 0 : last_row, cn, p.fast_rows, thread);
    TileFeed<float, CH, HT, K> dt32_feed(static_cast<const float *>(p.dt) + (p.dt_f32 ? c0 : 0), p.dt_st, p.dt_f32 ? last_row : 0, cn, p.fast_rows, thread);
    TileFeed<T, SP, HT, K> B_feed(static_cast<const T *>(p.B) + g * p.B_sg, p.B_st, last_row, (int)p.S, p.fast_vectors, thread),
        C_feed(static_cast<const T *>(p.Cm) + g * p.C_sg, p.C_st, last_row, (int)p.S, p.fast_vectors, thread);
    const float *entering = p.chunks + (at_rows.chunk + chunks - 1) * p.C * p.S + c0 * p.S;
    const int kept = cn * (int)p.S;
    auto bring = [&](int k) {  // chunk by chunk
      if (k < chunks) {
        const int rows = rows_of(k);
        const Stage s = stage(k);
        x_feed.bring(s.x, rows, cn, p.fast_rows, thread, -K);
        dy_feed.bring(s.dy, rows, cn, p.fast_rows, thread, -K);
        if (p.dt_f32) dt32_feed.bring(s.dt, rows, cn, p.fast_rows, thread, -K);
        else dt_feed.bring(s.dt, rows, cn, p.fast_rows, thread, -K);
        if (p.z) z_feed.bring(s.z, rows, cn, p.fast_rows, thread, -K);
        C_feed.bring(s.C, rows, (int)p.S, p.fast_vectors, thread, -K);
        if (!LOCAL) {
          B_feed.bring(s.B, rows, (int)p.S, p.fast_vectors, thread, -K);
          if (p.quad_states) {
            for (int q = thread * kQ; q < kept; q += HT * kQ) sm100::cp_async16(s.h + q, entering + q, 16u);
          } else {
            for (int q = thread; q < kept; q += HT) s.h[q] = entering[q];
          }
          entering -= p.C * p.S;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto form = [&](int k) {
      const Stage s = stage(k);
      const int at = (k & 1) * K, rows = rows_of(k);
      float2 v[ITEMS], x[ITEMS], d[ITEMS];
#pragma unroll
      for (int m = 0; m < ITEMS; ++m) {
        const int t = t0 + m * STEP, o = (K % STEP == 0 || t < K ? t : 0) * CH + c;
        v[m] = add2(p.dt_f32 ? load_pair<float>(s.dt, o) : load_pair<T>(s.dt, o), make_float2(bias[0], bias[1]));
        x[m] = load_pair<T>(s.x, o);
        d[m] = load_pair<T>(s.dy, o);
      }
      if (p.softplus)
#pragma unroll
        for (int m = 0; m < ITEMS; ++m) v[m] = softplus2(v[m]);
      if (p.z)
#pragma unroll
        for (int m = 0; m < ITEMS; ++m) {
          const int t = t0 + m * STEP;
          const float2 z = load_pair<T>(s.z, (K % STEP == 0 || t < K ? t : 0) * CH + c);
          d[m] = mul2(d[m], mul2(z, sigmoid2(z)));
        }
#pragma unroll
      for (int m = 0; m < ITEMS; ++m) {
        const int t = t0 + m * STEP;
        if (t >= rows) continue;
        const float2 in = mul2(v[m], x[m]);
        *reinterpret_cast<float4 *>(steps + (at + t) * CH + c) = make_float4(v[m].x, in.x, v[m].y, in.y);
        *reinterpret_cast<float2 *>(gs + (at + t) * CH + c) = d[m];
      }
#pragma unroll
      for (int q = Back::WIDEN ? thread * kQ : K * SP; q < K * SP; q += HT * kQ) {
        const float2 a0 = load_pair<T>(s.C, q), a1 = load_pair<T>(s.C, q + 2);
        *reinterpret_cast<float4 *>(Cs + at * SP + q) = make_float4(a0.x, a0.y, a1.x, a1.y);
        if (!LOCAL) {
          const float2 b0 = load_pair<T>(s.B, q), b1 = load_pair<T>(s.B, q + 2);
          *reinterpret_cast<float4 *>(Bs + at * SP + q) = make_float4(b0.x, b0.y, b1.x, b1.y);
        }
      }
    };
    auto put = [&](void *base, int64_t o, float2 v, auto type) {
      using V = decltype(type);
      V *to = static_cast<V *>(base) + o;
      if (p.pair_out) {
        if (c < cn) {
          if constexpr (sizeof(V) == 4) *reinterpret_cast<float2 *>(to) = v;
          else *reinterpret_cast<uint32_t *>(to) = narrow<V>(v);
        }
      } else {
        if (c < cn) to[0] = from_f32<V>(v.x);
        if (c + 1 < cn) to[1] = from_f32<V>(v.y);
      }
    };
    // Half a chunk's gradients: the parts of u, v, y and of dB and dC are added up, in a fixed order.
    auto finish = [&](int k, int half) {
      const Stage s = stage(k);
      const int at = (k & 1) * K, rows = rows_of(k);
      const int64_t row = first_row(k);
      const int t = half * HALF + thread / CP;
      if (thread < HALF * CP && t < rows) {
        float2 u = make_float2(0.f, 0.f), v = u, y = u;
#pragma unroll
        for (int j = 0; j < L; ++j) {
          u = add2(u, parts[part_of(t, 0, j, c / 2)]);
          v = add2(v, parts[part_of(t, 1, j, c / 2)]);
        }
        const int o = t * CH + c;
        const int64_t to = (row + t) * p.C + c0 + c;
        const float4 d = *reinterpret_cast<const float4 *>(steps + at * CH + o);
        const float2 gd = *reinterpret_cast<const float2 *>(gs + at * CH + o), x = load_pair<T>(s.x, o);
        put(p.dx, to, fma2(u, make_float2(d.x, d.z), mul2(gd, D)), T());
        float2 dt = fma2(v, both(kLn2), mul2(u, x));
        if (p.softplus) {
          const float2 w = add2(p.dt_f32 ? load_pair<float>(s.dt, o) : load_pair<T>(s.dt, o), make_float2(bias[0], bias[1]));
          dt = mul2(dt, sigmoid2(w));
        }
        if (p.dt_f32) put(p.ddt, to, dt, float());
        else put(p.ddt, to, dt, T());
        dD = fma2(gd, x, dD);
        dbias = add2(dt, dbias);
        if (p.z) {
#pragma unroll
          for (int j = 0; j < L; ++j) y = add2(y, parts[part_of(t, 2, j, c / 2)]);
          const float2 z = load_pair<T>(s.z, o), dy = load_pair<T>(s.dy, o);
          y = fma2(D, x, y);
          const float2 q = sigmoid2(z);
          put(p.dz, to, mul2(mul2(dy, y), mul2(q, fma2(z, fma2(q, both(-1.f), both(1.f)), both(1.f)))), T());
        }
      }
      // an item: four states of dB or dC of a token; where there are fewer than threads, two threads share one
      constexpr int OUT = HALF * 2 * L, SHARE = HT > OUT ? HT / OUT : 1, EACH = RT / L / SHARE;
#pragma unroll
      for (int m = thread / SHARE; m < OUT; m += HT / SHARE) {
        const int w = m / (2 * L), j = m % L, share = thread % SHARE;
        const float4 *from = sums + ((half * HALF + w) * 2 + m / L % 2) * RT + j;
        float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
        for (int r = 0; r < EACH; ++r) {
          const float4 v = from[(share * EACH + ((r + share) & (EACH - 1))) * L];
          a = add2(a, make_float2(v.x, v.y));
          b = add2(b, make_float2(v.z, v.w));
        }
#pragma unroll
        for (int r = 1; r < SHARE; r *= 2) {
          a = add2(a, make_float2(__shfl_xor_sync(0xffffffffu, a.x, r), __shfl_xor_sync(0xffffffffu, a.y, r)));
          b = add2(b, make_float2(__shfl_xor_sync(0xffffffffu, b.x, r), __shfl_xor_sync(0xffffffffu, b.y, r)));
        }
        if (share == 0 && half * HALF + w < rows)
          *reinterpret_cast<float4 *>(p.over_channels + ((int64_t)tile * p.p.T + row + half * HALF + w) * (2 * SP) + m % (2 * L) * kQ) =
              make_float4(a.x, a.y, b.x, b.y);
      }
    };
    auto meet = [&](bool all) {  // the feeding warps' copies (but the last group) have landed
      if (all) asm volatile("cp.async.wait_group 0;" ::: "memory");
      else asm volatile("cp.async.wait_group 1;" ::: "memory");
      asm volatile("bar.sync 1, %0;" ::"n"(HT) : "memory");
    };
    bring(0);
    bring(1);
    meet(false);
    if (chunks > 0) form(0);
    __syncthreads();
    for (int k = 0; k < chunks; ++k) {
      if (!LOCAL && k > 0) finish(k - 1, 0);  // while the running warps are at the chunk's second half
      __syncthreads();
      bring(k + 2);  // (where chunk k - 1 was)
      if (!LOCAL) finish(k, 1);
      meet(false);
      if (k + 1 < chunks) form(k + 1);
      if (!LOCAL && k % kSums == kSums - 1) add_up();
      __syncthreads();
    }
    if (!LOCAL && chunks > 0) finish(chunks - 1, 0);
    if (!LOCAL) add_up();
    meet(true);  // before the stages are used again
  }
  if (LOCAL) return;
  // dD and ddt_bias: a channel's rows are spread over the threads that share its number
  float4 *share = reinterpret_cast<float4 *>(ring);
  share[thread] = make_float4(total_D.x, total_D.y, total_bias.x, total_bias.y);
  asm volatile("bar.sync 1, %0;" ::"n"(HT) : "memory");
  if (thread < CP) {
    float4 v = share[thread];
    for (int k = 1; k < HT / CP; ++k) {
      const float4 o = share[k * CP + thread];
      v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
    }
    float *to = out + p.C * p.S + c0 + c;
    if (c < cn) to[0] = v.x, to[p.C] = v.z;
    if (c + 1 < cn) to[1] = v.y, to[p.C + 1] = v.w;
  }
}

// The gradients entering every piece of a sequence from behind, from those that the pieces pass on from zero.
template <int V>
__global__ void __launch_bounds__(kSsmThreads) gdp_ssm_join_back_kernel(const SsmProblem p) {
  const int64_t i = blockIdx.x, at = ((int64_t)blockIdx.y * kSsmThreads + threadIdx.x) * V, per = p.C * p.S;
  sm100::pdl_trigger();
  sm100::pdl_wait();
  if (at >= per) return;
  int64_t b, e;
  seq_rows(p.p, i, &b, &e);
  float S[V] = {}, A[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (p.dfin) S[k] = p.dfin[i * per + at + k];
    A[k] = p.A[at + k] * kLog2e;
  }
  if (b == e) {  // no piece will write the initial state's
    if (p.dinit)
#pragma unroll
      for (int k = 0; k < V; ++k) p.dinit[i * per + at + k] = S[k];
    return;
  }
  const int64_t r = b / p.piece + i, n = (e - b + p.piece - 1) / p.piece, c = at / p.S;
  float *enter = p.enter + r * per + at;
  const float *spans = p.spans + r * p.C + c;
  constexpr int AHEAD = 16;
  for (int64_t q = n - 1; q >= 0; q -= AHEAD) {
    float E[AHEAD][V], span[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (q - u > 0) {
        span[u] = spans[(q - u) * p.C];
        const Vec<float, V> v = load_vec<float, V>(enter + (q - u) * per);
#pragma unroll
        for (int k = 0; k < V; ++k) E[u][k] = v.v[k];
      }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (q - u >= 0) {
        store_vec<float, V>(enter + (q - u) * per, S);
        if (q - u > 0)
#pragma unroll
          for (int k = 0; k < V; ++k) S[k] = carry(S[k], E[u][k], A[k] * span[u]);
      }
  }
}

// dB and dC: the sums over the CTAs that share a group's channels, in their order, four states a thread; padding rows are
// zeros.
template <typename T>
__global__ void __launch_bounds__(256) gdp_ssm_vectors_kernel(const SsmProblem p, int SP) {
  const int quads = 2 * SP / kQ;
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x, row = k / quads, g = blockIdx.y;
  if (row >= p.p.T) return;
  const int q = (int)(k % quads) * kQ, state = q % SP;
  float2 a = make_float2(0.f, 0.f), b = a;
  if (row < cu_at(p.p, p.p.N)) {
    const float *from = p.over_channels + (g * p.tiles * p.p.T + row) * (2 * SP) + q;
#pragma unroll 8
    for (int i = 0; i < p.tiles; ++i, from += p.p.T * (2 * SP)) {
      const float4 v = *reinterpret_cast<const float4 *>(from);
      a = add2(a, make_float2(v.x, v.y));
      b = add2(b, make_float2(v.z, v.w));
    }
  }
  T *to = static_cast<T *>(q < SP ? p.dB : p.dC) + (row * p.G + g) * p.S + state;
  const float v[kQ] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int i = 0; i < kQ; ++i)
    if (state + i < p.S) to[i] = from_f32<T>(v[i]);
}

template <typename T, int L, bool FULL, bool LOCAL>
cudaError_t ssm_bwd(const SsmProblem &p, cudaStream_t stream) {
  using Back = SsmBack<T, L>;
  constexpr int most = Back::bytes(4, true);
  static_assert(most <= 227 * 1024, "fits an SM");
  const auto kernel = gdp_ssm_bwd_kernel<T, L, FULL, LOCAL>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  return gdp::launch_kernel(kernel, dim3((unsigned)((p.workers + (LOCAL ? 0 : 1)) * p.G * p.tiles)), dim3(kSsmFeed + kSsmThreads / 2),
                            Back::bytes(p.dt_f32 ? 4 : (int)sizeof(T), p.z != nullptr), stream, p.piece && !LOCAL, p);
}
template <typename T, int L>
cudaError_t ssm_bwd_by(const SsmProblem &p, cudaStream_t stream) {
  if (p.piece) {
    cudaError_t e = ssm_bwd<T, L, false, true>(p, stream);
    if (e != cudaSuccess) return e;
    const int64_t per = p.C * p.S, v = p.quad_states ? kQ : 1;
    const dim3 grid((unsigned)p.p.N, (unsigned)((per / v + kSsmThreads - 1) / kSsmThreads));
    e = gdp::launch_kernel(p.quad_states ? gdp_ssm_join_back_kernel<kQ> : gdp_ssm_join_back_kernel<1>, grid, dim3(kSsmThreads), 0, stream, true, p);
    if (e != cudaSuccess) return e;
  }
  return p.S == L * kQ ? ssm_bwd<T, L, true, false>(p, stream) : ssm_bwd<T, L, false, false>(p, stream);
}
template <typename T>
cudaError_t launch_ssm_bwd(const SsmProblem &p, cudaStream_t stream) {
  const int lanes = ssm_lanes(p.S), SP = lanes * kQ;
  cudaError_t e = lanes == 4 ? ssm_bwd_by<T, 4>(p, stream) : lanes == 8 ? ssm_bwd_by<T, 8>(p, stream) : ssm_bwd_by<T, 16>(p, stream);
  if (e != cudaSuccess || p.p.T == 0) return e;
  gdp_ssm_vectors_kernel<T><<<dim3((unsigned)((p.p.T * (2 * SP / kQ) + 255) / 256), (unsigned)p.G), 256, 0, stream>>>(p, SP);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace gdp
