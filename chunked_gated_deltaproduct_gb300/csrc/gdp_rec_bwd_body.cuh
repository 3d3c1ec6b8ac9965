// gdp_rec_bwd_body.cuh -- the backward scan of the gated linear recurrence (see gdp_rec_scan.cuh).
//
// With E_t = a_t D_t: D_t = d_output_t + E_{t+1} (the final state's gradient where a sequence ends),
// so a run of tokens maps the E that enters it from later tokens to A E + B, and the tiles go back in
// time.  dx and dg of a token need D_t, E_t and the state before the token, whose tile is the one of h
// (or of its 8-bit codes) shifted by a row.
#pragma once

#include <type_traits>

#include "gdp_rec_scan.cuh"

namespace gdp {
namespace layer {
namespace {

#ifndef SB8
#define SB8 0
#endif
constexpr int kBwdCtas = 2;  // resident CTAs per SM

template <typename TX, typename TG, int GATE, bool Q8, bool RAW>
struct BwdLayout {
  // tokens per warp: sixteen decays stay in registers, or eight with the input factors
  static constexpr int S = GATE == GDP_GATE_SIGMOID || sizeof(TX) == 4 || SB8 ? 8 : 16;
  static constexpr int kTile = kScanWarps * S;
  static constexpr bool kX = GATE == GDP_GATE_SIGMOID;
  static constexpr int g_off = 0, d_off = g_off + tile_bytes<TG>(kTile, RAW), h_off = d_off + tile_bytes<TX>(kTile, RAW);
  static constexpr int s_off = h_off + (Q8 ? tile_bytes<int8_t>(kTile, RAW) : tile_bytes<TX>(kTile, RAW));
  static constexpr int x_off = s_off + (Q8 ? kTile * 4 : 0), stage = (x_off + (kX ? tile_bytes<TX>(kTile, RAW) : 0) + 127) / 128 * 128;
  static constexpr int kStages = stage <= 22000 ? 4 : stage <= 34000 ? 3 : 2;
  static constexpr int kMeta = kStages + 1;
  static constexpr int parts = kStages * stage, enter = parts + Chain::parts_bytes, meta = enter + Chain::enter_bytes;
  static constexpr int bars = (meta + kMeta * (int)sizeof(TileMeta<S>) + 15) / 16 * 16;
  static constexpr int mail = (bars + (2 * kStages + Chain::bars) * 8 + 16 + 127) / 128 * 128;  // last: its size is the cluster's
};

struct BwdMaps {
  CUtensorMap g, dout, h, x;  // h: of the tensor or of the codes
};

template <typename TX, typename TG, int GATE, bool Q8, bool RAW>
__global__ void __launch_bounds__(kScanThreads, kBwdCtas) gdp_rec_bwd_scan_kernel(const __grid_constant__ BwdMaps maps, const RecBwd p) {
  using L = BwdLayout<TX, TG, GATE, Q8, RAW>;
  constexpr int S = L::S;
  extern __shared__ __align__(128) unsigned char smem[];
  TileMeta<S> *metas = reinterpret_cast<TileMeta<S> *>(smem + L::meta);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::bars), *empty = full + L::kStages;
  Chain ch;
  ch.parts = reinterpret_cast<float4 *>(smem + L::parts);
  ch.enter = reinterpret_cast<float2 *>(smem + L::enter);
  ch.mail = reinterpret_cast<float4 *>(smem + L::mail);
  ch.parts_full = empty + L::kStages;
  ch.enter_full = ch.parts_full + 1;
  ch.mail_full = ch.enter_full + 1;
  volatile int *gave_up = reinterpret_cast<volatile int *>(ch.mail_full + kMailSlots);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ScanShape &s = p.s;
  const int slice = (int)blockIdx.x / s.cluster, rank = (int)cluster_rank(), steps = (s.rows + s.cluster - 1) / s.cluster;
  const int64_t c0 = (int64_t)slice * kSlice;
  // checkpoint scales: the slice lies in one block of one row when a row is a multiple of 64 channels
  const bool one_scale = Q8 && p.group % kSlice == 0;
  const int64_t scales_per_token = Q8 ? s.C / p.group * p.blocks : 0;
  auto scale_index = [&](int64_t c) { return c / p.group * p.blocks + c % p.group / kBlock; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      sm100::mbar_init(&full[i], RAW || Q8 ? 33 : 1);
      sm100::mbar_init(&empty[i], kScanWarps);
    }
    sm100::mbar_init(ch.parts_full, kScanWarps);
    sm100::mbar_init(ch.enter_full, 1);
    for (int i = 0; i < kMailSlots; ++i) sm100::mbar_init(&ch.mail_full[i], 1);
    *gave_up = 0;
    sm100::mbar_init_fence();
  }
  __syncthreads();
  cluster_sync();  // the barriers stand before anyone posts to them

  if (warp == kLoadWarp) {
    const int64_t first = load_cu(s.cu, s.cu64, 0), end = min(load_cu(s.cu, s.cu64, s.N), s.T);
    SeqWindow win;
    win.load(s, max((int64_t)0, s.N - 32), lane);
    for (int n = 0; n < steps; ++n) {
      const int st = n % L::kStages, r = s.rows - 1 - (n * s.cluster + rank);
      const int64_t t0 = (int64_t)r * L::kTile;  // before row 0 in the last step of some CTAs: an empty tile
      TileMeta<S> &m = metas[n % L::kMeta];
      unsigned char *base = smem + st * L::stage;
      if (n >= L::kStages) ring_wait(&empty[st], (n / L::kStages + 1) & 1, gave_up, s.status, s.limit_ns);
      if (RAW) {
        load_words<TG>(base + L::g_off, p.g, t0, L::kTile, s.T, c0, s.C, lane);
        load_words<TX>(base + L::d_off, p.dout, t0, L::kTile, s.T, c0, s.C, lane);
        if (Q8) load_words<int8_t>(base + L::h_off, p.codes, t0 - 1, L::kTile, s.T, c0, s.C, lane);
        else load_words<TX>(base + L::h_off, p.h, t0 - 1, L::kTile, s.T, c0, s.C, lane);
        if (L::kX) load_words<TX>(base + L::x_off, p.x, t0, L::kTile, s.T, c0, s.C, lane);
      } else if (lane == 0) {
        mbar_expect_tx(&full[st], L::kTile * kSlice * (sizeof(TG) + (L::kX ? 2 : 1) * sizeof(TX) + (Q8 ? 1 : sizeof(TX))));
        sm100::tma_load_2d(base + L::g_off, &maps.g, (int)c0, (int)t0, &full[st]);
        sm100::tma_load_2d(base + L::d_off, &maps.dout, (int)c0, (int)t0, &full[st]);
        sm100::tma_load_2d(base + L::h_off, &maps.h, (int)c0, (int)t0 - 1, &full[st]);
        if (L::kX) sm100::tma_load_2d(base + L::x_off, &maps.x, (int)c0, (int)t0, &full[st]);
      }
      if (one_scale) {
        const int64_t at = scale_index(c0);
        for (int i = lane; i < L::kTile; i += 32) {
          const int64_t t = t0 - 1 + i;
          const bool in = t >= 0 && t < s.T;
          cp_async4(sm100::smem_u32(base + L::s_off + 4 * i), p.scales + (in ? t * scales_per_token + at : 0), in ? 4u : 0u);
        }
      }
      find_sequences<S, true>(s, m, win, t0, r + 1 == s.rows, c0, p.dfin, p.dinit, lane);
      if (lane == 0) {
        m.lo = (int)max((int64_t)0, min(first - t0, (int64_t)L::kTile));
        m.hi = (int)max((int64_t)0, min(end - t0, (int64_t)L::kTile));
      }
      __syncwarp();
      if (RAW || Q8) cp_async_arrive(&full[st]);
      if (lane == 0) sm100::mbar_arrive(&full[st]);
    }
    if (blockIdx.x == 0) check_sequences(s.cu, s.cu64, s.N, s.T, s.status, lane, 32);
  } else if (warp == kChainWarp) {
    chain_steps<S, L::kMeta, true>(s, ch, metas, steps, lane, gave_up);
  } else {
    const int64_t c = c0 + 2 * lane;
    const bool all_channels = c0 + kSlice <= s.C && p.vec_dx && p.vec_dg;
    const int64_t scale0 = Q8 ? scale_index(c) : 0, scale1 = Q8 ? scale_index(c + 1) : 0;
    const int block = kScanWarps - 1 - warp;  // this warp's tokens: rows block * S .. + S - 1, last first
    for (int n = 0; n < steps; ++n) {
      const int st = n % L::kStages;
      const unsigned char *base = smem + st * L::stage;
      const int64_t t0 = ((int64_t)s.rows - 1 - ((int64_t)n * s.cluster + rank)) * L::kTile + block * S;
      ring_wait(&full[st], (n / L::kStages) & 1, gave_up, s.status, s.limit_ns);
      const TileMeta<S> &m = metas[n % L::kMeta];
      const uint32_t starts = m.starts[block], ends = m.ends[block];
      const int lo = m.lo - block * S, hi = m.hi - block * S;
      auto row_of = [&](int off, int pitch, int i) { return base + off + (block * S + i) * pitch; };
      auto upstream = [&](int i) {
        return unpack<TX>(read_packed<TX, RAW>(base + L::d_off, block * S + i, lane, RAW ? raw_offset<TX>(p.dout, t0 + i, c0) : 0));
      };
      float2 a[S], f[L::kX ? S : 1];
      float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        float2 fi;
        gate_pair<GATE>(unpack<TG>(read_packed<TG, RAW>(base + L::g_off, block * S + i, lane, RAW ? raw_offset<TG>(p.g, t0 + i, c0) : 0)),
                        &a[i], &fi);
        if constexpr (L::kX) f[i] = fi;
        A = mul2(A, a[i]);
        B = mul2(a[i], add2(upstream(i), B));
      }
      if (ends) {  // again, token by token
        B = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
          if (ends >> i & 1u) B = read_state(p.dfin, m.end_row[block * S + i], s.C, c);
          B = mul2(a[i], add2(upstream(i), B));
        }
      }
      ch.parts[warp * 32 + lane] = make_float4(A.x, A.y, B.x, B.y);
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(ch.parts_full);
      ring_wait(ch.enter_full, n & 1, gave_up, s.status, s.limit_ns);
      float2 E = ch.enter[warp * 32 + lane];
      TX *dx = static_cast<TX *>(p.dx) + (t0 + S - 1) * s.C + c;
      TG *dg = static_cast<TG *>(p.dg) + (t0 + S - 1) * s.C + c;
      // the state before token i
      auto before = [&](int i) {
        if constexpr (Q8) {
          const unsigned char *q = row_of(L::h_off, tile_pitch<int8_t>(RAW), i) + (RAW ? raw_offset<int8_t>(p.codes, t0 + i - 1, c0) : 0) + 2 * lane;
          // a byte plus 128 under the exponent of 2^23 is 2^23 + 128 + code
          const uint32_t w = (RAW ? (uint32_t)q[0] | (uint32_t)q[1] << 8 : (uint32_t) * reinterpret_cast<const uint16_t *>(q)) ^ 0x8080u;
          const float2 v = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)), __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441))),
                                both(-8388736.f));
          if (one_scale) return mul2(v, both(*reinterpret_cast<const float *>(row_of(L::s_off, 4, i))));
          float2 sc = both(0.f);
          const int64_t t = t0 + i - 1;
          if (t >= 0 && t < s.T) {
            if (c < s.C) sc.x = p.scales[t * scales_per_token + scale0];
            if (c + 1 < s.C) sc.y = p.scales[t * scales_per_token + scale1];
          }
          return mul2(v, sc);
        } else {
          return unpack<TX>(read_packed<TX, RAW>(base + L::h_off, block * S + i, lane, RAW ? raw_offset<TX>(p.h, t0 + i - 1, c0) : 0));
        }
      };
      // D in, dx and dg out; E moves on to this token
      auto token = [&](int i, float2 prev, float2 *ox, float2 *og) {
        const float2 D = add2(upstream(i), E);
        E = mul2(a[i], D);
        if constexpr (L::kX) {
          const float2 in = unpack<TX>(read_packed<TX, RAW>(base + L::x_off, block * S + i, lane, RAW ? raw_offset<TX>(p.x, t0 + i, c0) : 0));
          *ox = mul2(f[i], D);
          *og = mul2(mul2(f[i], E), fma2(in, both(-1.f), prev));
        } else {
          *ox = D;
          *og = mul2(GATE == GDP_GATE_LOG ? E : D, prev);
        }
      };
      if (!(starts | ends) && lo <= 0 && hi >= S && all_channels) {
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
          float2 ox, og;
          token(i, before(i), &ox, &og);
          write_pair(dx, ox, true, true);
          write_pair(dg, og, true, true);
          dx -= s.C;
          dg -= s.C;
        }
      } else {
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
          if (ends >> i & 1u) E = read_state(p.dfin, m.end_row[block * S + i], s.C, c);
          float2 ox, og;
          token(i, starts >> i & 1u ? read_state(p.init, m.start_row[block * S + i], s.C, c) : before(i), &ox, &og);
          if (i >= lo && i < hi && c < s.C) {
            write_pair(dx, ox, c + 1 < s.C, p.vec_dx);
            write_pair(dg, og, c + 1 < s.C, p.vec_dg);
          }
          if (starts >> i & 1u) write_state(p.dinit, m.start_row[block * S + i], s.C, c, E);
          dx -= s.C;
          dg -= s.C;
        }
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&empty[st]);
    }
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another may still post to it
}

template <typename TX, typename TG, int GATE, bool Q8, bool RAW>
cudaError_t run_bwd_as(RecBwd &p, const BwdMaps &maps, cudaStream_t stream) {
  return launch_clusters(gdp_rec_bwd_scan_kernel<TX, TG, GATE, Q8, RAW>, p.s.slices, p.s.cluster,
                         BwdLayout<TX, TG, GATE, Q8, RAW>::mail + Chain::mail_bytes(p.s.cluster), stream, maps, p);
}

template <typename TX, typename TG, int GATE, bool Q8>
cudaError_t run_bwd(RecBwd &p, cudaStream_t stream) {
  using L = BwdLayout<TX, TG, GATE, Q8, false>;
  ScanShape &s = p.s;
  const int64_t rows = (s.T + L::kTile - 1) / L::kTile;
  s.rows = rows > 0 ? (int)rows : 1;
  s.slices = (int)((s.C + kSlice - 1) / kSlice);
  s.cluster = cluster_size(s.slices, s.rows, sm_count(), kBwdCtas);
  const RowSource &h = Q8 ? p.codes : p.h;
  constexpr int hs = Q8 ? 1 : (int)sizeof(TX);
  BwdMaps m;
  memset(&m, 0, sizeof(m));
  if (!tma_rows(p.g, sizeof(TG), s.T, s.C) || !tma_rows(p.dout, sizeof(TX), s.T, s.C) || !tma_rows(h, hs, s.T, s.C) ||
      (L::kX && !tma_rows(p.x, sizeof(TX), s.T, s.C)))
    return run_bwd_as<TX, TG, GATE, Q8, true>(p, m, stream);
  cudaError_t e;
  if ((e = tmap_matrix(&m.g, p.g.base, s.T, s.C, p.g.stride * sizeof(TG), sizeof(TG), kSlice, L::kTile)) != cudaSuccess) return e;
  if ((e = tmap_matrix(&m.dout, p.dout.base, s.T, s.C, p.dout.stride * sizeof(TX), sizeof(TX), kSlice, L::kTile)) != cudaSuccess) return e;
  if ((e = tmap_matrix(&m.h, h.base, s.T, s.C, h.stride * hs, hs, kSlice, L::kTile)) != cudaSuccess) return e;
  if (L::kX && (e = tmap_matrix(&m.x, p.x.base, s.T, s.C, p.x.stride * sizeof(TX), sizeof(TX), kSlice, L::kTile)) != cudaSuccess) return e;
  return run_bwd_as<TX, TG, GATE, Q8, false>(p, m, stream);
}

template <typename TX, typename TG, int GATE>
cudaError_t run_bwd_saved(RecBwd &p, cudaStream_t stream) {
  return p.codes.base ? run_bwd<TX, TG, GATE, true>(p, stream) : run_bwd<TX, TG, GATE, false>(p, stream);
}

}  // namespace

template <typename TX, typename TG>
cudaError_t launch_rec_bwd(RecBwd &p, int gate, cudaStream_t stream) {
  if (gate == GDP_GATE_LOG) return run_bwd_saved<TX, TG, GDP_GATE_LOG>(p, stream);
  if (gate == GDP_GATE_ALPHA) return run_bwd_saved<TX, TG, GDP_GATE_ALPHA>(p, stream);
  return run_bwd_saved<TX, TG, GDP_GATE_SIGMOID>(p, stream);
}

}  // namespace layer
}  // namespace gdp
