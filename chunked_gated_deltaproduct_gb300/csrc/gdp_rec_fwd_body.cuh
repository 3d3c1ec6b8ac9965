// gdp_rec_fwd_body.cuh -- the forward scan of the gated linear recurrence (see gdp_rec_scan.cuh).
#pragma once

#include "gdp_rec_scan.cuh"

namespace gdp {
namespace layer {
namespace {

constexpr int kFwdCtas = 2;  // resident CTAs per SM

template <typename TX, typename TG, bool RAW>
struct FwdLayout {
  static constexpr int S = 8;  // tokens per warp
  static constexpr int kTile = kScanWarps * S;
  static constexpr int x_off = 0, g_off = tile_bytes<TX>(kTile, RAW), stage = g_off + tile_bytes<TG>(kTile, RAW);
  static constexpr int kStages = stage <= 18000 ? 4 : stage <= 26000 ? 3 : 2;
  static constexpr int kMeta = kStages + 1;
  static constexpr int parts = kStages * stage, enter = parts + Chain::parts_bytes, meta = enter + Chain::enter_bytes;
  static constexpr int bars = (meta + kMeta * (int)sizeof(TileMeta<S>) + 15) / 16 * 16;
  static constexpr int mail = (bars + (2 * kStages + Chain::bars) * 8 + 16 + 127) / 128 * 128;  // last: its size is the cluster's
};

template <typename TX, typename TG, int GATE, bool RAW>
__global__ void __launch_bounds__(kScanThreads, kFwdCtas)
    gdp_rec_fwd_scan_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g, const RecFwd p) {
  using L = FwdLayout<TX, TG, RAW>;
  constexpr int S = L::S;
  extern __shared__ __align__(128) unsigned char smem[];
  TileMeta<S> *metas = reinterpret_cast<TileMeta<S> *>(smem + L::meta);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::bars), *empty = full + L::kStages;
  Chain ch;
  ch.parts = reinterpret_cast<float4 *>(smem + L::parts);
  ch.enter = reinterpret_cast<float2 *>(smem + L::enter);
  ch.mail = reinterpret_cast<float4 *>(smem + L::mail);
  ch.parts_full = empty + L::kStages;
  ch.enter_full = ch.parts_full + 2;
  ch.mail_full = ch.enter_full + 2;
  volatile int *gave_up = reinterpret_cast<volatile int *>(ch.mail_full + kMailSlots);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ScanShape &s = p.s;
  const int slice = (int)blockIdx.x / s.cluster, rank = (int)cluster_rank(), steps = (s.rows + s.cluster - 1) / s.cluster;
  const int64_t c0 = (int64_t)slice * kSlice;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      sm100::mbar_init(&full[i], RAW ? 33 : 1);
      sm100::mbar_init(&empty[i], kScanWarps);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&ch.parts_full[i], kScanWarps);
      sm100::mbar_init(&ch.enter_full[i], 1);
    }
    for (int i = 0; i < kMailSlots; ++i) sm100::mbar_init(&ch.mail_full[i], 1);
    *gave_up = 0;
    sm100::mbar_init_fence();
  }
  __syncthreads();
  cluster_sync();  // the barriers stand before anyone posts to them

  if (warp == kLoadWarp) {
    const int64_t first = load_cu(s.cu, s.cu64, 0), end = min(load_cu(s.cu, s.cu64, s.N), s.T);
    for (int n = 0; n < steps; ++n) {
      const int st = n % L::kStages, r = n * s.cluster + rank;
      const int64_t t0 = (int64_t)r * L::kTile;
      TileMeta<S> &m = metas[n % L::kMeta];
      unsigned char *base = smem + st * L::stage;
      if (n >= L::kStages) ring_wait(&empty[st], (n / L::kStages + 1) & 1, gave_up, s.status, s.limit_ns);
      if (RAW) {
        load_words<TX>(base + L::x_off, p.x, t0, L::kTile, s.T, c0, s.C, lane);
        load_words<TG>(base + L::g_off, p.g, t0, L::kTile, s.T, c0, s.C, lane);
      } else if (lane == 0) {
        mbar_expect_tx(&full[st], L::kTile * kSlice * (sizeof(TX) + sizeof(TG)));
        sm100::tma_load_2d(base + L::x_off, &map_x, (int)c0, (int)t0, &full[st]);
        sm100::tma_load_2d(base + L::g_off, &map_g, (int)c0, (int)t0, &full[st]);
      }
      find_sequences<S>(s, m, t0, r + 1 == s.rows, c0, p.from, s.slots ? nullptr : p.to, lane);
      if (lane == 0) {
        m.lo = (int)max((int64_t)0, min(first - t0, (int64_t)L::kTile));
        m.hi = (int)max((int64_t)0, min(end - t0, (int64_t)L::kTile));
      }
      __syncwarp();
      if (RAW) cp_async_arrive(&full[st]);
      if (lane == 0) sm100::mbar_arrive(&full[st]);
    }
    if (blockIdx.x == 0) check_sequences(s.cu, s.cu64, s.N, s.T, s.status, lane, 32);
  } else if (warp == kPostWarp) {
    post_steps<S, L::kMeta>(s, ch, metas, steps, lane, gave_up);
  } else if (warp == kFoldWarp) {
    fold_steps<S, L::kMeta>(s, ch, metas, steps, lane, gave_up);
  } else {
    const int64_t c = c0 + 2 * lane;
    // decay and input of token i (of this warp's S) of the tile in stage st
    auto token = [&](int st, int64_t t0, int i, float2 *a, float2 *b) {
      const unsigned char *base = smem + st * L::stage;
      const float2 x = read_pair<TX, RAW>(base + L::x_off, warp * S + i, lane, RAW ? raw_offset<TX>(p.x, t0 + i, c0) : 0);
      const float2 g = read_pair<TG, RAW>(base + L::g_off, warp * S + i, lane, RAW ? raw_offset<TG>(p.g, t0 + i, c0) : 0);
      float2 f;
      gate_eval<GATE>(g.x, &a->x, &f.x);
      gate_eval<GATE>(g.y, &a->y, &f.y);
      *b = GATE == GDP_GATE_SIGMOID ? make_float2(f.x * x.x, f.y * x.y) : x;
    };
    auto x_offset = [&](int64_t t0, int i) { return RAW ? raw_offset<TX>(p.x, t0 + i, c0) : 0; };
    auto g_offset = [&](int64_t t0, int i) { return RAW ? raw_offset<TG>(p.g, t0 + i, c0) : 0; };
    auto keep = [&](int st, int64_t t0, int i, float2 v) {
      put_bits<TX, RAW>(smem + st * L::stage + L::x_off, warp * S + i, lane, x_offset(t0, i), v.x);
      put_bits<TG, RAW>(smem + st * L::stage + L::g_off, warp * S + i, lane, g_offset(t0, i), v.y);
    };
    auto kept = [&](int st, int64_t t0, int i) {
      return make_float2(get_bits<TX, RAW>(smem + st * L::stage + L::x_off, warp * S + i, lane, x_offset(t0, i)),
                         get_bits<TG, RAW>(smem + st * L::stage + L::g_off, warp * S + i, lane, g_offset(t0, i)));
    };
    for (int n = 0; n <= steps; ++n) {
      if (n < steps) {  // tile n from zero
        const int st = n % L::kStages;
        ring_wait(&full[st], (n / L::kStages) & 1, gave_up, s.status, s.limit_ns);
        const TileMeta<S> &m = metas[n % L::kMeta];
        const int64_t t0 = ((int64_t)n * s.cluster + rank) * L::kTile + warp * S;
        const uint32_t starts = m.starts[warp];
        float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < S; ++i) {
          float2 a, b;
          token(st, t0, i, &a, &b);
          const bool start = starts >> i & 1u;
          if (start) B = read_state(p.from, m.start_row[warp * S + i], s.C, c);
          B = make_float2(fmaf(a.x, B.x, b.x), fmaf(a.y, B.y, b.y));
          // the state after a sequence's first token takes the place of that token's x and g: its
          // incoming state may be overwritten (in place, by the warp that ends the sequence) before
          // this warp comes back to the tile
          if (start) keep(st, t0, i, B);
          A = make_float2(A.x * a.x, A.y * a.y);
        }
        ch.parts[((n & 1) * kScanWarps + warp) * 32 + lane] = make_float4(A.x, A.y, B.x, B.y);
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&ch.parts_full[n & 1]);
      }
      if (n > 0) {  // tile n - 1 from its entering state
        const int q = n - 1, st = q % L::kStages;
        const TileMeta<S> &m = metas[q % L::kMeta];
        const int64_t t0 = ((int64_t)q * s.cluster + rank) * L::kTile + warp * S;
        const uint32_t starts = m.starts[warp], ends = m.ends[warp];
        const int lo = m.lo - warp * S, hi = m.hi - warp * S;
        ring_wait(&ch.enter_full[q & 1], (q >> 1) & 1, gave_up, s.status, s.limit_ns);
        float2 h = ch.enter[((q & 1) * kScanWarps + warp) * 32 + lane];
        TX *out = static_cast<TX *>(p.h) + t0 * s.C + c;
#pragma unroll
        for (int i = 0; i < S; ++i) {
          float2 a, b;
          token(st, t0, i, &a, &b);
          h = make_float2(fmaf(a.x, h.x, b.x), fmaf(a.y, h.y, b.y));
          if (starts >> i & 1u) h = kept(st, t0, i);
          if (i >= lo && i < hi && c < s.C) write_pair(out, h, c + 1 < s.C, p.vec_out);
          if (ends >> i & 1u) write_state(p.to, m.end_row[warp * S + i], s.C, c, h);
          out += s.C;
        }
        if (starts) sm100::fence_async_smem();  // what keep() wrote, before the next tile's copy
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&empty[st]);
      }
    }
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another may still post to it
}

template <typename TX, typename TG, int GATE, bool RAW>
cudaError_t run_fwd_as(RecFwd &p, const CUtensorMap *maps, cudaStream_t stream) {
  return launch_clusters(gdp_rec_fwd_scan_kernel<TX, TG, GATE, RAW>, p.s.slices, p.s.cluster,
                         FwdLayout<TX, TG, RAW>::mail + Chain::mail_bytes(p.s.cluster), stream, maps[0], maps[1], p);
}

template <typename TX, typename TG, int GATE>
cudaError_t run_fwd(RecFwd &p, cudaStream_t stream) {
  using L = FwdLayout<TX, TG, false>;
  ScanShape &s = p.s;
  const int64_t rows = (s.T + L::kTile - 1) / L::kTile;
  s.rows = rows > 0 ? (int)rows : 1;
  s.slices = (int)((s.C + kSlice - 1) / kSlice);
  s.cluster = cluster_size(s.slices, s.rows, sm_count(), kFwdCtas);
  CUtensorMap maps[2];
  memset(maps, 0, sizeof(maps));
  auto fits = [&](const RowSource &src, size_t es) { return s.T > 0 && s.C >= kSlice && aligned(src.base, 16) && src.stride * es % 16 == 0; };
  s.raw = !(fits(p.x, sizeof(TX)) && fits(p.g, sizeof(TG)));
  cudaError_t e = cudaSuccess;
  if (!s.raw) {
    if ((e = tmap_matrix(&maps[0], p.x.base, s.T, s.C, p.x.stride * sizeof(TX), sizeof(TX), kSlice, L::kTile)) != cudaSuccess) return e;
    if ((e = tmap_matrix(&maps[1], p.g.base, s.T, s.C, p.g.stride * sizeof(TG), sizeof(TG), kSlice, L::kTile)) != cudaSuccess) return e;
  }
  return s.raw ? run_fwd_as<TX, TG, GATE, true>(p, maps, stream) : run_fwd_as<TX, TG, GATE, false>(p, maps, stream);
}

template <typename TX, typename TG>
cudaError_t run_fwd_gate(RecFwd &p, int gate, cudaStream_t stream) {
  if (gate == GDP_GATE_LOG) return run_fwd<TX, TG, GDP_GATE_LOG>(p, stream);
  if (gate == GDP_GATE_ALPHA) return run_fwd<TX, TG, GDP_GATE_ALPHA>(p, stream);
  return run_fwd<TX, TG, GDP_GATE_SIGMOID>(p, stream);
}

}  // namespace
}  // namespace layer
}  // namespace gdp
