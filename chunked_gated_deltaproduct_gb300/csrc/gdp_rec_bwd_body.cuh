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

constexpr int kBwdCtas = 2;  // resident CTAs per SM

template <typename TX, typename TG, int GATE, bool Q8, bool RAW>
struct BwdLayout {
  // Bytes of a channel and token; three stages where that leaves ten tokens per warp, else two (when it was
  // chosen, 65536 x 4096 from codes: 401 us with three, 448 us with two; 8 x 4096 x 2048 sigmoid: 174 us and 154 us).
  static constexpr int kBytes = (int)(sizeof(TG) + sizeof(TX) * (GATE == GDP_GATE_SIGMOID ? 2 : 1) + (Q8 ? 1 : sizeof(TX)));
  static constexpr int kStages = scan_tokens(3 * kBytes) >= 10 ? 3 : 2, S = scan_tokens(kStages * kBytes);
  static constexpr int kTile = kScanWarps * S;
  static constexpr bool kX = GATE == GDP_GATE_SIGMOID;
  static constexpr int g_off = 0, d_off = g_off + tile_bytes<TG>(kTile, RAW), h_off = d_off + tile_bytes<TX>(kTile, RAW);
  static constexpr int s_off = h_off + (Q8 ? tile_bytes<int8_t>(kTile, RAW) : tile_bytes<TX>(kTile, RAW));
  static constexpr int x_off = s_off + (Q8 ? (kTile * 4 + 127) / 128 * 128 : 0);
  static constexpr int stage = x_off + (kX ? tile_bytes<TX>(kTile, RAW) : 0);
  static constexpr int kMeta = kStages + 1;
  static constexpr bool kShortWaits = true;
  static constexpr int parts = kStages * stage, parts_m = parts + Chain::parts_bytes, parts_e = parts_m + Chain::parts_m_bytes, enter = parts_e + Chain::parts_e_bytes, meta = enter + Chain::enter_bytes;
  static constexpr int bars = (meta + kMeta * (int)sizeof(TileMeta<S>) + 15) / 16 * 16;
  static constexpr int mail = (bars + (2 * kStages + Chain::bars) * 8 + 16 + 127) / 128 * 128;  // last: its size is the cluster's
  // TMA destinations, 16-byte arrays, barriers, and the largest cluster's whole
  static_assert(g_off % 128 == 0 && d_off % 128 == 0 && h_off % 128 == 0 && x_off % 128 == 0 && s_off % 4 == 0 && S * kSlice * sizeof(TX) % 128 == 0 && S * kSlice * sizeof(TG) % 128 == 0 && stage % 128 == 0, "TMA reads and writes at 128-byte boundaries");
  static_assert(parts % 16 == 0 && parts_m % 8 == 0 && parts_e % 4 == 0 && enter % 16 == 0 && meta % 4 == 0 && bars % 8 == 0 && mail % 16 == 0, "alignment");
  static_assert(mail + Chain::mail_bytes(RAW ? 8 : 16) <= kScanSmem && mail + Chain::mail_bytes(16) <= 227 * 1024, "two CTAs per SM");
};

struct BwdMaps {
  CUtensorMap g, dout, h, x;  // h: of the tensor or of the codes
  CUtensorMap dx, dg;
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
  // checkpoint scales: the slice lies in one block of one row when a row is a multiple of 64 channels, or all
  const bool one_scale = Q8 && (p.group % kSlice == 0 || p.group == s.C);
  const int64_t scales_per_token = Q8 ? s.C / p.group * p.blocks : 0;
  auto scale_index = [&](int64_t c) { return c / p.group * p.blocks + c % p.group / kBlock; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      sm100::mbar_init(&full[i], RAW || Q8 ? 33 : 1);
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
    win.load(s, max((int64_t)0, s.N - 32), lane);
    int n = 0;
    for (; n < steps; ++n) {
      const int st = n % L::kStages, r = s.rows - 1 - (n * s.cluster + rank);
      const int64_t t0 = (int64_t)r * L::kTile;  // before row 0 in the last step of some CTAs: an empty tile
      TileMeta<S> &m = metas[n % L::kMeta];
      unsigned char *base = smem + st * L::stage;
      if (n >= L::kStages && !ring_wait<L::kShortWaits>(&empty[st], (n / L::kStages + 1) & 1, gave_up, s.status, s.limit_ns)) break;
      if (RAW) {
        load_rows<TG>(base + L::g_off, p.g, t0, L::kTile, s.T, c0, s.C, lane);
        load_rows<TX>(base + L::d_off, p.dout, t0, L::kTile, s.T, c0, s.C, lane);
        if (Q8) load_rows<int8_t>(base + L::h_off, p.codes, t0 - 1, L::kTile, s.T, c0, s.C, lane);
        else load_rows<TX>(base + L::h_off, p.h, t0 - 1, L::kTile, s.T, c0, s.C, lane);
        if (L::kX) load_rows<TX>(base + L::x_off, p.x, t0, L::kTile, s.T, c0, s.C, lane);
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
      if (t0 + L::kTile > end && t0 >= 0) {
        zero_rows_of<TX>(p.dx, max(end, t0), min(s.T, t0 + L::kTile), s.C, c0, lane);
        zero_rows_of<TG>(p.dg, max(end, t0), min(s.T, t0 + L::kTile), s.C, c0, lane);
      }
      __syncwarp();
      if (RAW || Q8) cp_async_arrive(&full[st]);
      if (lane == 0) sm100::mbar_arrive(&full[st]);
    }
    if (*gave_up) drain_loads<L::kStages>(full, n, RAW || Q8);
    if (blockIdx.x == 0) check_sequences(s.cu, s.cu64, s.N, s.T, s.status, lane, 32);
  } else if (warp == kChainWarp) {
    chain_steps<S, L::kMeta, L::kShortWaits>(s, ch, metas, steps, lane, gave_up);
  } else {
    const int64_t c = c0 + 2 * lane;
    // dx and dg take the places of d_output and g in the stage and leave by TMA stores (each warp its own
    // rows), so that a warp does not wait for memory to take them; rows of unaligned outputs, and tiles with
    // rows of no sequence, do not
    const bool bulk = !RAW && p.vec_out;
    const int64_t scale0 = Q8 ? scale_index(c) : 0, scale1 = Q8 ? scale_index(c + 1) : 0;
    const int block = kScanWarps - 1 - warp;  // this warp's tokens: rows block * S .. + S - 1, last first
    for (int n = 0; n < steps; ++n) {
      const int st = n % L::kStages;
      const unsigned char *base = smem + st * L::stage;
      const int64_t t0 = ((int64_t)s.rows - 1 - ((int64_t)n * s.cluster + rank)) * L::kTile + block * S;
      if (!ring_wait<L::kShortWaits>(&full[st], (n / L::kStages) & 1, gave_up, s.status, s.limit_ns)) break;
      const TileMeta<S> &m = metas[n % L::kMeta];
      const uint32_t starts = m.starts[block], ends = m.ends[block];
      const int lo = m.lo - block * S, hi = m.hi - block * S;
      auto row_of = [&](int off, int pitch, int i) { return base + off + (block * S + i) * pitch; };
      auto upstream = [&](int i) {
        return unpack<TX>(read_packed<TX, RAW>(base + L::d_off, block * S + i, lane, RAW ? raw_offset<TX>(p.dout, t0 + i, c0) : 0));
      };
      float2 kept[S];  // gates
      float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
      LargestGate<TG, GATE> largest;
#pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        const auto g = read_packed<TG, RAW>(base + L::g_off, block * S + i, lane, RAW ? raw_offset<TG>(p.g, t0 + i, c0) : 0);
        largest.see(g);
        kept[i] = gate_kept<GATE>(unpack<TG>(g));
        float2 f;
        const float2 a = gate_decay<GATE>(kept[i], &f);
        A = mul2(A, a);
        B = mul2(a, add2(upstream(i), B));
      }
      if (ends) {  // again, token by token
        A = both(1.f);
        keep_only<S>(kept);
        B = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
          if (ends >> i & 1u) B = read_state(p.dfin, m.end_row[block * S + i], s.C, c);
          float2 f;
          B = mul2(gate_decay<GATE>(kept[i], &f), add2(upstream(i), B));
        }
      }
      const bool unsafe = write_part(ch, warp * 32 + lane, A, B, largest, ends != 0u);
      __syncwarp();
      if (lane == 0) {
        sm100::mbar_arrive(ch.parts_full);
        if (n > 0) {  // the last tile's stage, once its stores have read it
          sm100::bulk_wait_read<0>();
          sm100::mbar_arrive(&empty[(n - 1) % L::kStages]);
        }
      }
      if (unsafe) {
        float2 *products = ch.parts_m + warp * 32 + lane;
        int *exponents = ch.parts_e + warp * 32 + lane;
        if (largest.holds(A)) {
          *products = A;
          *exponents = 0;
        } else {
          write_products<TG, GATE, RAW, S>(products, exponents, base + L::g_off, block * S, lane, p.g, t0, c0);
        }
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(ch.products_full);
      if (!ring_wait<L::kShortWaits>(ch.enter_full, n & 1, gave_up, s.status, s.limit_ns)) break;
      keep_only<S>(kept);
      float2 E = ch.enter[warp * 32 + lane];
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
      // Four tokens' inputs are read before any of their outputs is written (outputs go to the same shared
      // memory, so that the compiler keeps the order: token by token the second run took 221 cycles each).
      // whole: every row belongs to a sequence and the outputs leave by TMA; plain: no sequence begins or ends
      auto run = [&](auto whole_, auto plain_) {
        constexpr bool kWhole = decltype(whole_)::value, kPlain = decltype(plain_)::value;
        TX *dx = static_cast<TX *>(p.dx) + (t0 + S - 1) * s.C + c;
        TG *dg = static_cast<TG *>(p.dg) + (t0 + S - 1) * s.C + c;
        TX *dx_rows = reinterpret_cast<TX *>(smem + st * L::stage + L::d_off) + block * S * kSlice + 2 * lane;
        TG *dg_rows = reinterpret_cast<TG *>(smem + st * L::stage + L::g_off) + block * S * kSlice + 2 * lane;
#pragma unroll
        for (int hi4 = S - 1; hi4 >= 0; hi4 -= 4) {
          float2 up[4], prev[4], in[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = hi4 - u;
            if (i < 0) break;
            up[u] = upstream(i);
            prev[u] = !kPlain && (starts >> i & 1u) ? read_state(p.init, m.start_row[block * S + i], s.C, c) : before(i);
            if constexpr (L::kX)
              in[u] = unpack<TX>(read_packed<TX, RAW>(base + L::x_off, block * S + i, lane, RAW ? raw_offset<TX>(p.x, t0 + i, c0) : 0));
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = hi4 - u;
            if (i < 0) break;
            if (!kPlain && (ends >> i & 1u)) E = read_state(p.dfin, m.end_row[block * S + i], s.C, c);
            float2 f;
            const float2 a = gate_decay<GATE>(kept[i], &f), D = add2(up[u], E);
            E = mul2(a, D);
            float2 ox = D, og;
            if constexpr (L::kX) {
              ox = mul2(f, D);
              og = mul2(mul2(f, E), fma2(in[u], both(-1.f), prev[u]));
            } else {
              og = mul2(GATE == GDP_GATE_LOG ? E : D, prev[u]);
            }
            if constexpr (kWhole) {
              write_pair(dx_rows + i * kSlice, ox, true, true);
              write_pair(dg_rows + i * kSlice, og, true, true);
            } else if (i >= lo && i < hi && c < s.C) {
              write_pair(dx, ox, c + 1 < s.C, p.pair_dx);
              write_pair(dg, og, c + 1 < s.C, p.pair_dg);
            }
            dx -= s.C;
            dg -= s.C;
            if (!kPlain && (starts >> i & 1u)) write_state(p.dinit, m.start_row[block * S + i], s.C, c, E);
          }
        }
        if constexpr (kWhole) {
          sm100::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            sm100::tma_store_2d(&maps.dx, dx_rows, (int)c0, (int)t0);
            sm100::tma_store_2d(&maps.dg, dg_rows, (int)c0, (int)t0);
            sm100::bulk_commit();
          }
        }
      };
      const bool whole = lo <= 0 && hi >= S && bulk;
      if (!RAW && whole && !(starts | ends)) run(std::true_type{}, std::true_type{});
      else if (!RAW && whole) run(std::true_type{}, std::false_type{});
      else run(std::false_type{}, std::false_type{});
      __syncwarp();
    }
    if (lane == 0) sm100::bulk_wait_all();
  }
  leave_cluster(gave_up);
}

template <typename TX, typename TG, int GATE, bool Q8, bool RAW>
cudaError_t run_bwd_as(const RecBwd &p, const BwdMaps &maps, cudaStream_t stream) {
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
  p.vec_out = tma_rows(RowSource{p.dx, s.C}, sizeof(TX), s.T, s.C) && tma_rows(RowSource{p.dg, s.C}, sizeof(TG), s.T, s.C);
  if (p.vec_out) {
    if ((e = tmap_matrix(&m.dx, p.dx, s.T, s.C, s.C * sizeof(TX), sizeof(TX), kSlice, L::S)) != cudaSuccess) return e;
    if ((e = tmap_matrix(&m.dg, p.dg, s.T, s.C, s.C * sizeof(TG), sizeof(TG), kSlice, L::S)) != cudaSuccess) return e;
  }
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
