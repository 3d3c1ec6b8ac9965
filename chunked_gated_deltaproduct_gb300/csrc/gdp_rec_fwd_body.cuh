// gdp_rec_fwd_body.cuh -- the forward scan of the gated linear recurrence (see gdp_rec_scan.cuh).
#pragma once

#include <type_traits>

#include "gdp_rec_scan.cuh"

namespace gdp {
namespace layer {
namespace {

constexpr int kFwdCtas = 2;  // resident CTAs per SM

template <typename TX, typename TG, int GATE, bool RAW>
struct FwdLayout {
  // Sigmoid gates: decays and inputs (three special-function operations a channel to form again) stay in
  // registers, and the stage is free after the first run; else the second run reads the inputs again
  // (at 65536 x 4096 bf16, when it was chosen: 262 us; with three stages 322 us).
  static constexpr bool kKeep = GATE == GDP_GATE_SIGMOID;
  static constexpr int kStages = 2;
  static constexpr int S = scan_tokens(kStages * (int)(sizeof(TX) + sizeof(TG)) + (int)sizeof(TX));
  static constexpr int kTile = kScanWarps * S;
  static constexpr int x_off = 0, g_off = tile_bytes<TX>(kTile, RAW), stage = g_off + tile_bytes<TG>(kTile, RAW);
  static constexpr int kMeta = kStages + 1;
  static constexpr bool kShortWaits = !kKeep;
  static constexpr int out = kStages * stage, out_bytes = RAW ? 0 : kTile * kSlice * (int)sizeof(TX);
  static constexpr int parts = out + out_bytes, parts_m = parts + Chain::parts_bytes, parts_e = parts_m + Chain::parts_m_bytes, enter = parts_e + Chain::parts_e_bytes, meta = enter + Chain::enter_bytes;
  static constexpr int bars = (meta + kMeta * (int)sizeof(TileMeta<S>) + 15) / 16 * 16;
  static constexpr int mail = (bars + (2 * kStages + Chain::bars) * 8 + 16 + 127) / 128 * 128;  // last: its size is the cluster's
  // TMA destinations, 16-byte arrays, barriers, and the largest cluster's whole
  static_assert(x_off % 128 == 0 && g_off % 128 == 0 && out % 128 == 0 && S * kSlice * sizeof(TX) % 128 == 0 && stage % 128 == 0, "TMA writes to 128-byte boundaries");
  static_assert(parts % 16 == 0 && parts_m % 8 == 0 && parts_e % 4 == 0 && enter % 16 == 0 && meta % 4 == 0 && bars % 8 == 0 && mail % 16 == 0, "alignment");
  static_assert(mail + Chain::mail_bytes(RAW ? 8 : 16) <= kScanSmem && mail + Chain::mail_bytes(16) <= 227 * 1024, "two CTAs per SM");
};

template <typename TX, typename TG, int GATE, bool RAW>
__global__ void __launch_bounds__(kScanThreads, kFwdCtas)
    gdp_rec_fwd_scan_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
                            const __grid_constant__ CUtensorMap map_h, const RecFwd p) {
  using L = FwdLayout<TX, TG, GATE, RAW>;
  constexpr int S = L::S;
  extern __shared__ __align__(128) unsigned char smem[];
  TileMeta<S> *metas = reinterpret_cast<TileMeta<S> *>(smem + L::meta);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::bars), *empty = full + L::kStages;
  Chain ch;
  ch.parts = reinterpret_cast<float4 *>(smem + L::parts);
  ch.parts_m = reinterpret_cast<float2 *>(smem + L::parts_m);
  ch.parts_e = reinterpret_cast<int *>(smem + L::parts_e);
  ch.enter = reinterpret_cast<float2 *>(smem + L::enter);
  ch.mail = reinterpret_cast<float4 *>(smem + L::mail);
  ch.wide_mail = reinterpret_cast<int2 *>(ch.mail + kMailSlots * p.s.cluster * 32);
  ch.parts_full = empty + L::kStages;
  ch.products_full = ch.parts_full + 1;
  ch.enter_full = ch.products_full + 1;
  ch.wide_full = ch.enter_full + 1;
  ch.mail_full = ch.wide_full + 1;
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
    sm100::mbar_init(ch.parts_full, kScanWarps);
    sm100::mbar_init(ch.products_full, kScanWarps);
    sm100::mbar_init(ch.enter_full, 1);
    sm100::mbar_init(ch.wide_full, 1);
    for (int i = 0; i < kMailSlots; ++i) sm100::mbar_init(&ch.mail_full[i], 1);
    *gave_up = 0;
    sm100::mbar_init_fence();
  }
  __syncthreads();
  cluster_sync();  // the barriers stand before anyone posts to them

  if (warp == kLoadWarp) {
    // rows [first, end) belong to sequences, whatever cu_seqlens hold: nothing outside [0, T) is written
    const int64_t first = clamp_row(load_cu(s.cu, s.cu64, 0), s.T), end = clamp_row(load_cu(s.cu, s.cu64, s.N), s.T);
    SeqWindow win;
    win.load(s, 0, lane);
    int n = 0;
    for (; n < steps; ++n) {
      const int st = n % L::kStages, r = n * s.cluster + rank;
      const int64_t t0 = (int64_t)r * L::kTile;
      TileMeta<S> &m = metas[n % L::kMeta];
      unsigned char *base = smem + st * L::stage;
      if (n >= L::kStages && !ring_wait<L::kShortWaits>(&empty[st], (n / L::kStages + 1) & 1, gave_up, s.status, s.limit_ns)) break;
      if (RAW) {
        load_rows<TX>(base + L::x_off, p.x, t0, L::kTile, s.T, c0, s.C, lane);
        load_rows<TG>(base + L::g_off, p.g, t0, L::kTile, s.T, c0, s.C, lane);
      } else if (lane == 0) {
        mbar_expect_tx(&full[st], L::kTile * kSlice * (sizeof(TX) + sizeof(TG)));
        sm100::tma_load_2d(base + L::x_off, &map_x, (int)c0, (int)t0, &full[st]);
        sm100::tma_load_2d(base + L::g_off, &map_g, (int)c0, (int)t0, &full[st]);
      }
      find_sequences<S, false>(s, m, win, t0, r + 1 == s.rows, c0, p.from, s.slots ? nullptr : p.to, lane);
      if (lane == 0) {
        m.lo = (int)max((int64_t)0, min(first - t0, (int64_t)L::kTile));
        m.hi = (int)max((int64_t)0, min(end - t0, (int64_t)L::kTile));
      }
      if (s.zero_pad && t0 + L::kTile > end) zero_rows_of<TX>(p.h, max(end, t0), min(s.T, t0 + L::kTile), s.C, c0, lane);
      __syncwarp();
      if (RAW) cp_async_arrive(&full[st]);
      if (lane == 0) sm100::mbar_arrive(&full[st]);
    }
    if (*gave_up) drain_loads<L::kStages>(full, n, RAW);
    if (blockIdx.x == 0) check_sequences(s.cu, s.cu64, s.N, s.T, s.status, lane, 32);
  } else if (warp == kChainWarp) {
    chain_steps<S, L::kMeta, L::kShortWaits>(s, ch, metas, steps, lane, gave_up);
  } else {
    const int64_t c = c0 + 2 * lane;
    // outputs leave through shared memory and TMA stores (each warp its own rows), so that a warp does not
    // wait for memory to take them; rows of unaligned outputs, and tiles with rows of no sequence, do not
    const bool bulk = !RAW && p.vec_out;
    unsigned char *mine = smem + L::out + warp * S * kSlice * (int)sizeof(TX);
    for (int n = 0; n < steps; ++n) {
      const int st = n % L::kStages;
      const unsigned char *xs = smem + st * L::stage + L::x_off, *gs = smem + st * L::stage + L::g_off;
      const int64_t t0 = ((int64_t)n * s.cluster + rank) * L::kTile + warp * S;
      if (!ring_wait<L::kShortWaits>(&full[st], (n / L::kStages) & 1, gave_up, s.status, s.limit_ns)) break;
      const TileMeta<S> &m = metas[n % L::kMeta];
      const uint32_t starts = m.starts[warp], ends = m.ends[warp];
      const int lo = m.lo - warp * S, hi = m.hi - warp * S;
      // ---- from zero: the decays stay in registers, and the inputs too (kKeep).  Where a sequence begins,
      // the decay's place takes the state after that token.
      float2 a[S], b[L::kKeep ? S : 1];
      float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
      LargestGate<TG, GATE> largest;
      auto read_x = [&](int i) {
        return unpack<TX>(read_packed<TX, RAW>(xs, warp * S + i, lane, RAW ? raw_offset<TX>(p.x, t0 + i, c0) : 0));
      };
#pragma unroll
      for (int i = 0; i < S; ++i) {
        float2 f;
        const auto g = read_packed<TG, RAW>(gs, warp * S + i, lane, RAW ? raw_offset<TG>(p.g, t0 + i, c0) : 0);
        largest.see(g);
        a[i] = gate_decay<GATE>(gate_kept<GATE>(unpack<TG>(g)), &f);
        const float2 x = GATE == GDP_GATE_SIGMOID ? mul2(f, read_x(i)) : read_x(i);
        if constexpr (L::kKeep) b[i] = x;
        B = fma2(a[i], B, x);
        A = mul2(A, a[i]);
      }
      if (starts) {  // again, token by token
        A = both(1.f);
        keep_only<S>(a);
        B = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < S; ++i) {
          if (starts >> i & 1u) B = read_state(p.from, m.start_row[warp * S + i], s.C, c);
          float2 x;
          if constexpr (L::kKeep) x = b[i];
          else x = read_x(i);
          B = fma2(a[i], B, x);
          if (starts >> i & 1u) a[i] = B;
        }
      }
      const bool unsafe = write_part(ch, warp * 32 + lane, A, B, largest, starts != 0u);
      __syncwarp();
      if (lane == 0) {
        sm100::mbar_arrive(ch.parts_full);
        sm100::bulk_wait_read<0>();  // the last tile's store has read `mine`
      }
      if (unsafe) {
        float2 *products = ch.parts_m + warp * 32 + lane;
        int *exponents = ch.parts_e + warp * 32 + lane;
        if (largest.holds(A)) {
          *products = A;
          *exponents = 0;
        } else {
          write_products<TG, GATE, RAW, S>(products, exponents, gs, warp * S, lane, p.g, t0, c0);
        }
      }
      __syncwarp();
      if (lane == 0) {
        sm100::mbar_arrive(ch.products_full);
        if (L::kKeep) sm100::mbar_arrive(&empty[st]);
      }
      if (!ring_wait<L::kShortWaits>(ch.enter_full, n & 1, gave_up, s.status, s.limit_ns)) break;
      keep_only<S>(a);
      // ---- from the entering state.  Four tokens' inputs are read before their outputs are written (the
      // compiler keeps the order of accesses to shared memory).
      // whole: every row belongs to a sequence and the outputs leave by TMA; plain: no sequence begins or ends
      float2 h = ch.enter[warp * 32 + lane];
      auto run = [&](auto whole_, auto plain_) {
        constexpr bool kWhole = decltype(whole_)::value, kPlain = decltype(plain_)::value;
        TX *out = static_cast<TX *>(p.h) + t0 * s.C + c, *rows = reinterpret_cast<TX *>(mine) + 2 * lane;
#pragma unroll
        for (int lo4 = 0; lo4 < S; lo4 += 4) {
          float2 x[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (lo4 + u >= S) break;
            if constexpr (L::kKeep) x[u] = b[lo4 + u];
            else x[u] = read_x(lo4 + u);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = lo4 + u;
            if (i >= S) break;
            h = !kPlain && (starts >> i & 1u) ? a[i] : fma2(a[i], h, x[u]);
            if constexpr (kWhole) write_pair(rows + i * kSlice, h, true, true);
            else if (i >= lo && i < hi && c < s.C) write_pair(out, h, c + 1 < s.C, p.pair_out);
            out += s.C;
            if (!kPlain && (ends >> i & 1u)) write_state(p.to, m.end_row[warp * S + i], s.C, c, h);
          }
        }
        if constexpr (kWhole) {
          sm100::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            sm100::tma_store_2d(&map_h, mine, (int)c0, (int)t0);
            sm100::bulk_commit();
          }
        }
      };
      const bool whole = lo <= 0 && hi >= S && bulk;
      if (!RAW && whole && !(starts | ends)) run(std::true_type{}, std::true_type{});
      else if (!RAW && whole) run(std::true_type{}, std::false_type{});
      else run(std::false_type{}, std::false_type{});
      if (!L::kKeep) {
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&empty[st]);
      }
    }
    if (lane == 0) sm100::bulk_wait_all();
  }
  leave_cluster(gave_up);
}

template <typename TX, typename TG, int GATE, bool RAW>
cudaError_t run_fwd_as(const RecFwd &p, const CUtensorMap *maps, cudaStream_t stream) {
  return launch_clusters(gdp_rec_fwd_scan_kernel<TX, TG, GATE, RAW>, p.s.slices, p.s.cluster,
                         FwdLayout<TX, TG, GATE, RAW>::mail + Chain::mail_bytes(p.s.cluster), stream, maps[0], maps[1], maps[2], p);
}

template <typename TX, typename TG, int GATE>
cudaError_t run_fwd(RecFwd &p, cudaStream_t stream) {
  using L = FwdLayout<TX, TG, GATE, false>;
  ScanShape &s = p.s;
  const int64_t rows = (s.T + L::kTile - 1) / L::kTile;
  s.rows = rows > 0 ? (int)rows : 1;
  s.slices = (int)((s.C + kSlice - 1) / kSlice);
  s.cluster = cluster_size(s.slices, s.rows, sm_count(), kFwdCtas);
  CUtensorMap maps[3];
  memset(maps, 0, sizeof(maps));
  if (!tma_rows(p.x, sizeof(TX), s.T, s.C) || !tma_rows(p.g, sizeof(TG), s.T, s.C)) return run_fwd_as<TX, TG, GATE, true>(p, maps, stream);
  cudaError_t e;
  if ((e = tmap_matrix(&maps[0], p.x.base, s.T, s.C, p.x.stride * sizeof(TX), sizeof(TX), kSlice, L::kTile)) != cudaSuccess) return e;
  if ((e = tmap_matrix(&maps[1], p.g.base, s.T, s.C, p.g.stride * sizeof(TG), sizeof(TG), kSlice, L::kTile)) != cudaSuccess) return e;
  p.vec_out = tma_rows(RowSource{p.h, s.C}, sizeof(TX), s.T, s.C);
  if (p.vec_out && (e = tmap_matrix(&maps[2], p.h, s.T, s.C, s.C * sizeof(TX), sizeof(TX), kSlice, L::S)) != cudaSuccess) return e;
  return run_fwd_as<TX, TG, GATE, false>(p, maps, stream);
}

}  // namespace

template <typename TX, typename TG>
cudaError_t launch_rec_fwd(RecFwd &p, int gate, cudaStream_t stream) {
  if (gate == GDP_GATE_LOG) return run_fwd<TX, TG, GDP_GATE_LOG>(p, stream);
  if (gate == GDP_GATE_ALPHA) return run_fwd<TX, TG, GDP_GATE_ALPHA>(p, stream);
  return run_fwd<TX, TG, GDP_GATE_SIGMOID>(p, stream);
}

}  // namespace layer
}  // namespace gdp
