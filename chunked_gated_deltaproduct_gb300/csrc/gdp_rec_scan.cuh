// gdp_rec_scan.cuh -- what the forward and the backward kernel of the gated linear recurrence share.
//
// A run of tokens maps the entering state h to A h + B (A the product of its decays, B its end state
// from zero), so tiles of time are worked on side by side.  The packed rows [0, T) are cut into tiles
// of 8 S tokens x 64 channels whatever the sequences' lengths (a sequence's first token simply
// replaces the state).  A cluster of CTAs owns 64 channels for all of time: in step n its CTA k works
// on tile n * cluster + k.  In a CTA,
//   - a loading warp brings tiles ahead into a ring of shared-memory stages (TMA boxes, or 16-byte
//     asynchronous copies where rows are not 16-byte aligned) and finds the sequences in them;
//   - eight warps of S tokens each run the tile from zero, which gives each warp's (A, B), keep what
//     is dear to form again in registers (see the layouts), and run it again from their entering states;
//   - a chaining warp folds the eight (A, B) in between, writes the tile's (A, B) into every CTA of the
//     cluster (distributed shared memory, completing on the reader's barrier) and takes the cluster's
//     tiles in order of time from the state it carries: the eight entering states, and the state that
//     enters the next step.
// Every value comes from the same operations in the same order on every run.  Nothing of the chain passes
// through global memory: with (A, B) and states published there a hop took 5 us, which 6.8 TB/s would have to
// cover with 34 MB of waiting tiles (1.97 ms at 65536 x 4096 bf16, now 0.27 ms).  Every wait is bounded.
//
// Bound: memory (a multiply-add and an exponential per element against 6 or 9 bytes).  At 65536 x 4096 bf16 the
// forward moves 1.61 GB in 265 us (6.1 TB/s), the backward from 8-bit states 2.42 GB in 432 us (5.6 TB/s); at
// smaller sizes the latency of a step (load, run, chain, run) bounds: 2.1 us at 65536 x 4096 (128 steps), 2.5 us
// where sequences begin and end inside the tiles (64 packed requests x 2048, 83 steps).  Of that, keeping products of
// decays within range (below) costs 2 to 6 % (261, 412 and 201 us without, and with wrong results for some gates).
#pragma once

#include <climits>
#include <type_traits>

#include <cuda.h>

#include "gdp_layer.cuh"
#include "gdp_sm100.cuh"

namespace gdp {
namespace layer {

constexpr int kSlice = 64;        // channels of a tile: two per lane
constexpr int kScanWarps = 8;     // warps that compute
constexpr int kLoadWarp = kScanWarps, kChainWarp = kScanWarps + 1;
constexpr int kScanThreads = 32 * (kScanWarps + 2);
constexpr int kMailSlots = 2;     // steps whose posts may be under way at once (see chain_steps)

struct ScanShape {
  const void *cu;
  int cu64;
  int64_t T, N, C;
  int rows, slices;  // tiles in time and in channels
  const int32_t *slots;
  int64_t num_slots;
  uint32_t *status;
  int cluster;       // CTAs that share a slice's channels
  uint64_t limit_ns;
  int withhold;      // test of the failure path: the first tile's (A, B) is not posted
  int zero_pad;      // rows in [cu_seqlens[N], T) are written as zeros
};

// Sequences of one tile, found by the loading warp.
template <int S>
struct TileMeta {
  int lo, hi;                     // rows of the tile that belong to sequences
  uint32_t fresh;                 // bit w: in the chain's w-th warp a sequence begins (going back in time: ends)
  uint32_t starts[kScanWarps], ends[kScanWarps];  // per warp: its tokens that begin / end a sequence
  int start_row[kScanWarps * S], end_row[kScanWarps * S];  // state row of that sequence, -1: none
};

template <typename T>
constexpr int tile_pitch(bool raw) { return kSlice * (int)sizeof(T) + (raw ? 16 : 0); }
// One input tensor [T][C]: its address for the word-wise copies.
struct RowSource {
  const void *base;
  int64_t stride;  // elements
};
// Whether TMA can fetch its tiles.
inline bool tma_rows(const RowSource &src, size_t elem, int64_t T, int64_t C) {
  return T > 0 && C >= kSlice && aligned(src.base, 16) && src.stride * elem % 16 == 0;
}
// Bytes a tensor's tile takes in a stage.
template <typename T>
constexpr int tile_bytes(int rows, bool raw) { return (rows * tile_pitch<T>(raw) + 127) / 128 * 128; }

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(sm100::smem_u32(bar)), "r"(bytes) : "memory");
}

// Whole warp: rows [t0, t0 + rows) x channels [c0, c0 + 64) of a tensor whose rows start anywhere, by
// asynchronous copies of the 16-byte words that hold them; a row keeps its offset within its first word
// (raw_offset).  The words' other bytes belong to neighbouring rows: nothing before the tensor's first
// element's 4-byte word or after its last element is read.  Rows outside [0, T) become zeros.  Tiles away from
// the tensor's first and last rows go eight rows at a time without a check per word, the others word by word
// (everywhere so: 308 us at 16384 x 4095; a bulk copy per row: 298 us).
template <typename T>
__device__ __forceinline__ void load_rows(unsigned char *tile, const RowSource &src, int64_t t0, int rows, int64_t T_, int64_t c0,
                                          int64_t C, int lane) {
  constexpr int kWords = tile_pitch<T>(true) / 16;
  const int64_t pitch = src.stride * (int64_t)sizeof(T);
  if (t0 >= 1 && t0 + rows < T_ && pitch >= 16 * kWords + 16) {  // every word lies between two rows of the tensor
    const int q = lane & 3;
    int r = lane >> 2;
    uintptr_t at = reinterpret_cast<uintptr_t>(src.base) + (uintptr_t)((t0 + r) * pitch + c0 * (int64_t)sizeof(T));
    unsigned char *to = tile + r * tile_pitch<T>(true) + 16 * q;
#pragma unroll 2
    for (; r < rows; r += 8, at += 8 * pitch, to += 8 * tile_pitch<T>(true)) {
      const unsigned char *from = reinterpret_cast<const unsigned char *>(at & ~(uintptr_t)15) + 16 * q;
#pragma unroll
      for (int k = 0; k < kWords; k += 4)
        if (k + 4 <= kWords || q < kWords - k) sm100::cp_async16(to + 16 * k, from + 16 * k, 16u);
    }
    return;
  }
  const uint32_t wanted = (uint32_t)min((int64_t)kSlice, C - c0) * (uint32_t)sizeof(T);
  const uintptr_t base = reinterpret_cast<uintptr_t>(src.base);
  const uintptr_t end = base + (uintptr_t)(((T_ - 1) * src.stride + C) * (int64_t)sizeof(T));
  for (int i = lane; i < rows * kWords; i += 32) {
    const int r = i / kWords, w = i % kWords;
    const int64_t t = t0 + r;
    const bool in = t >= 0 && t < T_;
    const uintptr_t at = base + (uintptr_t)(((in ? t : 0) * src.stride + c0) * (int64_t)sizeof(T));
    const uintptr_t word = (at & ~(uintptr_t)15) + 16u * w;
    unsigned char *to = tile + r * tile_pitch<T>(true) + 16 * w;
    if (!in || word >= at + wanted) {
      sm100::cp_async16(to, reinterpret_cast<const void *>(base & ~(uintptr_t)15), 0u);  // zeros, nothing is read
    } else if (word >= base) {
      sm100::cp_async16(to, reinterpret_cast<const void *>(word), (uint32_t)min((uintptr_t)16, end - word));
    } else {  // the tensor begins within this word
      for (uintptr_t b = base & ~(uintptr_t)3; b < word + 16 && b < end; b += 4)
        cp_async4(sm100::smem_u32(to + (b - word)), reinterpret_cast<const void *>(b), (uint32_t)min((uintptr_t)4, end - b));
    }
  }
}
// Offset of row t's first channel within its first 16-byte word.
template <typename T>
__device__ __forceinline__ int raw_offset(const RowSource &src, int64_t t, int64_t c0) {
  return (int)((reinterpret_cast<uintptr_t>(src.base) + (uintptr_t)((t * src.stride + c0) * (int64_t)sizeof(T))) & 15u);
}

// The pair as it is stored: 16-bit types packed in one register.
template <typename T>
struct Packed {
  using type = uint32_t;
};
template <>
struct Packed<float> {
  using type = float2;
};
template <typename T, bool RAW>
__device__ __forceinline__ typename Packed<T>::type read_packed(const unsigned char *tile, int r, int lane, int offset) {
  if constexpr (sizeof(T) == 4) {
    const float *p = reinterpret_cast<const float *>(tile + r * tile_pitch<T>(RAW) + offset) + 2 * lane;
    if constexpr (RAW) return make_float2(p[0], p[1]);
    else return *reinterpret_cast<const float2 *>(p);
  } else if constexpr (RAW) {
    const uint16_t *p = reinterpret_cast<const uint16_t *>(tile + r * tile_pitch<T>(true) + offset) + 2 * lane;
    return (uint32_t)p[0] | (uint32_t)p[1] << 16;
  } else {
    return *reinterpret_cast<const uint32_t *>(tile + r * tile_pitch<T>(false) + lane * 4);
  }
}
template <typename T>
__device__ __forceinline__ float2 unpack(typename Packed<T>::type v) {
  if constexpr (sizeof(T) == 4) {
    return v;
  } else if constexpr (sizeof(T) == 2) {
    return widen<T>(v);
  }
}

// Both channels' gates in two steps: what stays in registers between the two runs over a tile (the decay;
// for the sigmoid e^-g, held to 2^125, from which either half follows to its own relative precision: the decay
// stays above 2^-125, next to the end of fp32, and the factor is 1), and decay and input factor from it.
template <int GATE>
__device__ __forceinline__ float2 gate_kept(float2 g) {
  if constexpr (GATE == GDP_GATE_ALPHA) return g;
  float2 t = mul2(g, both(GATE == GDP_GATE_LOG ? kLog2e : -kLog2e));
  if constexpr (GATE == GDP_GATE_SIGMOID) {
    asm("min.NaN.f32 %0, %0, 0f42FA0000;" : "+f"(t.x));
    asm("min.NaN.f32 %0, %0, 0f42FA0000;" : "+f"(t.y));
  }
  return make_float2(ex2(t.x), ex2(t.y));
}
template <int GATE>
__device__ __forceinline__ float2 gate_decay(float2 kept, float2 *f) {
  if constexpr (GATE != GDP_GATE_SIGMOID) {
    *f = both(1.f);
    return kept;
  } else {
    const float2 d = add2(kept, both(1.f)), a = make_float2(rcp(d.x), rcp(d.y));
    *f = mul2(kept, a);
    return a;
  }
}
// Makes another run over the tile form decay and factor from these again, and read the tile again (the
// compiler would keep what the run before formed and read, and spill).
template <int S>
__device__ __forceinline__ void keep_only(float2 *kept) {
#pragma unroll
  for (int i = 0; i < S; ++i) asm volatile("" : "+f"(kept[i].x), "+f"(kept[i].y)::"memory");
}
// Tokens per warp when a channel and token takes `bytes` of shared memory (all stages and the outputs), so
// that with the chain's part two CTAs share an SM; at most sixteen gates of two channels stay in registers.
constexpr int scan_tokens(int bytes) {
  const int n = 160 / bytes / 2 * 2;
  return n > 16 ? 16 : n;
}
constexpr int kScanSmem = 113 * 1024 + 512 - 1024;  // of a CTA, two per SM

template <typename T>
__device__ __forceinline__ void write_pair(T *p, float2 v, bool two, bool vec) {
  if (vec) {  // even channel count, aligned base: one store
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float2 *>(p) = v;
    } else {
      *reinterpret_cast<uint32_t *>(p) = narrow<T>(v);
    }
  } else {
    if (sizeof(T) == 2 && two && (reinterpret_cast<uintptr_t>(p) & 3u) == 0) {
      *reinterpret_cast<uint32_t *>(p) = narrow<T>(v);
    } else {
      p[0] = from_f32<T>(v.x);
      if (two) p[1] = from_f32<T>(v.y);
    }
  }
}
// The lane's two channels of a state row (channels past C read as zero / are not written).
__device__ __forceinline__ float2 read_state(const float *p, int row, int64_t C, int64_t c) {
  if (!p || row < 0) return make_float2(0.f, 0.f);
  const float *q = p + (int64_t)row * C + c;
  return make_float2(c < C ? q[0] : 0.f, c + 1 < C ? q[1] : 0.f);
}
__device__ __forceinline__ void write_state(float *p, int row, int64_t C, int64_t c, float2 v) {
  if (!p || row < 0) return;
  float *q = p + (int64_t)row * C + c;
  if (c < C) q[0] = v.x;
  if (c + 1 < C) q[1] = v.y;
}

// 32 consecutive sequences, one per lane of the loading warp, kept from tile to tile (a CTA's tiles
// go one way in time), so that a tile inside a long sequence costs no access to cu_seqlens.
struct SeqWindow {
  int64_t base, b, e;  // lane: bounds of sequence base + lane (past N: both beyond any row)
  bool ok;
  __device__ __forceinline__ void load(const ScanShape &p, int64_t at, int lane) {
    base = at;
    b = e = INT64_MAX;
    ok = false;
    if (base + lane < p.N) {
      b = load_cu(p.cu, p.cu64, base + lane);
      e = load_cu(p.cu, p.cu64, base + lane + 1);
      ok = b >= 0 && b <= e && e <= p.T;
    }
  }
  __device__ __forceinline__ int64_t first_begin() const { return __shfl_sync(0xffffffffu, b, 0); }
  __device__ __forceinline__ int64_t last_end() const { return __shfl_sync(0xffffffffu, e, 31); }
};

// Whole warp: the first i in [lo, hi] with i == hi or cu[i] >= t, 32 probes a round.
__device__ __forceinline__ int64_t first_at_least(const ScanShape &p, int64_t lo, int64_t hi, int64_t t, int lane) {
  while (lo < hi) {
    const int64_t chunk = (hi - lo + 31) / 32, at = lo + (lane + 1) * chunk - 1;
    const uint32_t hit = __ballot_sync(0xffffffffu, at >= hi || load_cu(p.cu, p.cu64, at) >= t);
    const int f = hit ? __ffs(hit) - 1 : 32;
    hi = min(hi, lo + (f + 1) * chunk - 1);
    lo = min(hi, lo + f * chunk);
  }
  return lo;
}

// Whole warp: the sequences that begin or end in tile rows [t0, t0 + 8 S), into m; those without
// tokens at a position in the tile (or at T, for the last tile in time) pass their state from `from`
// to `to` right away.  REV: the CTA's tiles go back in time.
template <int S, bool REV>
__device__ __forceinline__ void find_sequences(const ScanShape &p, TileMeta<S> &m, SeqWindow &win, int64_t t0, bool last, int64_t c0,
                                               const float *from, float *to, int lane) {
  constexpr int kTile = kScanWarps * S;
  const int64_t t1 = t0 + kTile;
  if (lane < kScanWarps) m.starts[lane] = m.ends[lane] = 0u;
  __syncwarp();
  if (!REV && win.base + 32 < p.N && win.last_end() < t0)  // on to the first sequence that ends at or after t0
    win.load(p, first_at_least(p, win.base + 32, p.N, t0, lane) - 1, lane);
  if (REV && win.base > 0 && win.first_begin() >= t1)  // back to the last ones that begin before t1
    win.load(p, max((int64_t)0, first_at_least(p, 0, win.base, t1, lane) - 32), lane);
  for (;;) {
    const int64_t b = win.b, e = win.e;
    const bool begins = win.ok && b < e && b >= t0 && b < t1, ends = win.ok && b < e && e > t0 && e <= t1;
    const bool none = win.ok && b == e && b >= t0 && (b < t1 || last);
    if (__any_sync(0xffffffffu, begins || ends || none)) {
      int row = (int)win.base + lane;
      if (p.slots && (begins || ends || none)) {
        row = p.slots[win.base + lane];
        if (row < -1 || row >= p.num_slots) {
          if (c0 == 0) set_status(p.status, GDP_DEV_ERR_SLOT);
          row = -1;
        }
      }
      if (begins) {
        m.start_row[b - t0] = row;
        atomicOr(&m.starts[(b - t0) / S], 1u << ((b - t0) % S));
      }
      if (ends) {
        m.end_row[e - 1 - t0] = row;
        atomicOr(&m.ends[(e - 1 - t0) / S], 1u << ((e - 1 - t0) % S));
      }
      if (to) {
        for (uint32_t left = __ballot_sync(0xffffffffu, none); left; left &= left - 1) {
          const int at = (int)win.base + __ffs(left) - 1;
          write_state(to, at, p.C, c0 + 2 * lane, read_state(from, at, p.C, c0 + 2 * lane));
        }
      }
    }
    if (!REV) {
      if (win.base + 32 >= p.N || (!last && win.last_end() >= t1)) break;
      win.load(p, win.base + 32, lane);
    } else {
      if (win.base == 0 || win.first_begin() < t0) break;
      win.load(p, max((int64_t)0, win.base - 32), lane);
    }
  }
  __syncwarp();
  const uint32_t cuts = lane < kScanWarps ? (REV ? m.ends[kScanWarps - 1 - lane] : m.starts[lane]) : 0u;
  const uint32_t fresh = __ballot_sync(0xffffffffu, cuts != 0u);
  if (lane == 0) m.fresh = fresh;
}

// An entry of cu_seqlens as a row: within [0, T], so that a tile's place relative to it cannot overflow.
__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t T) { return max((int64_t)0, min(v, T)); }

// Whole warp (the loading one, which has time): zeros into rows [from, to) of an output, channels [c0, c0 + 64).  The
// rows are padding, which the computing warps do not write (zeros written by them cost 2 to 5 % of a backward without
// padding, 419 and 430 against 411 us at 65536 x 4096 from codes).
template <typename T>
__device__ __forceinline__ void zero_rows_of(void *out, int64_t from, int64_t to, int64_t C, int64_t c0, int lane) {
  const int64_t c = c0 + 2 * lane;
#pragma unroll 1
  for (T *at = static_cast<T *>(out) + from * C + c; from < to; ++from, at += C) {
    if (c < C) at[0] = from_f32<T>(0.f);
    if (c + 1 < C) at[1] = from_f32<T>(0.f);
  }
}

// cu_seqlens ascending from 0 to at most T (any number of threads, `first` of `step`).
__device__ __forceinline__ void check_sequences(const void *cu, int cu64, int64_t N, int64_t T, uint32_t *status, int64_t first,
                                                int64_t step) {
  for (int64_t s = first; s < N; s += step) {
    const int64_t b = load_cu(cu, cu64, s), e = load_cu(cu, cu64, s + 1);
    if (b > e || b < 0 || e > T || (s == 0 && b != 0)) set_status(status, GDP_DEV_ERR_CU_SEQLENS);
  }
}

// ---- products of decays beyond fp32 ----
// A run's product A of decays may leave fp32's range though no state does: decays of 2 over 128 tokens while the
// state is zero, decays of 0.4 under an infinite state, a rise and its undoing.  The definition never forms such a
// product.  A plain product is right where no decay is above 2^(1/16), so that a tile's rises by 2^8 at most, and it
// ends above 2^-118, so that no part of it was below 2^-126; and where it ends below that it is right enough for a
// state of at most 2^16 (it is off by 2^8 times 2^-149, the state by 2^-125).  Everything else goes as A 2^e: with
// e = 0 and A plain where the whole is a normal number, else with A in [1, 2) in magnitude (a decay of exactly
// zero, infinity or NaN: itself, e = 0).  Which form a channel's product takes depends on its own tokens and state,
// and not on what its neighbours need.
constexpr float kNormal = 0x1p-126f, kMost = 0x1.fffffep127f;  // fp32's normal numbers
constexpr float kSafe = 0x1p-118f, kLargeState = 0x1p16f;

// v as m 2^e with 1 <= |m| < 2; zero, infinity and NaN are themselves (e = 0).
__device__ __forceinline__ float split(float v, int &e) {
  e = 0;
  uint32_t b = __float_as_uint(v);
  if ((b & 0x7fffffffu) == 0u || (b & 0x7f800000u) == 0x7f800000u) return v;
  if ((b & 0x7f800000u) == 0u) {
    b = __float_as_uint(v * 0x1p24f);
    e = -24;
  }
  e += (int)(b >> 23 & 255u) - 127;
  return __uint_as_float((b & 0x807fffffu) | 0x3f800000u);
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ bool outside(float A) { return !(fabsf(A) >= kNormal && fabsf(A) <= kMost); }
struct WideProduct {
  float m;  // a product of numbers of split (up to 16 before settle)
  int e;
  __device__ __forceinline__ void times(float v, int k) {  // by v 2^k
    int i;
    m *= split(v, i);
    e += i + k;
  }
  __device__ __forceinline__ void settle() {
    int i;
    m = split(m, i);
    e = outside(m) ? 0 : e + i;
    if (e >= -126 && e <= 127) {
      m *= power2(e);
      e = 0;
    }
  }
};
__device__ __forceinline__ int pack_exponents(int x, int y) { return (x & 0xffff) | y << 16; }
__device__ __forceinline__ int low_exponent(int v) { return (int)(short)(v & 0xffff); }
__device__ __forceinline__ int high_exponent(int v) { return v >> 16; }
// A 2^e as it is used: two factors, applied one after the other, so that only the result can leave the range (beyond
// 2^-252 and 2^254 any normal state gives zero or infinity alike).
struct Factors {
  float a, b;
  __device__ __forceinline__ Factors(float A, int e) {
    e = max(-252, min(e, 254));
    a = A * power2(e / 2);
    b = power2(e - e / 2);
  }
  __device__ __forceinline__ float apply(float h, float add) const { return b == 1.f ? fmaf(a, h, add) : fmaf(a * h, b, add); }
};
// A 2^e in 32 bits, a sign, nine bits of exponent and 22 of fraction: half a unit is 2^-23 of a product that has
// itself been rounded as often as it has factors.  Only products below 2^-118 or beyond fp32 are read back from it.
__device__ __forceinline__ uint32_t wide_code(float A, int e) {
  const uint32_t b = __float_as_uint(A);
  if (outside(A)) return A == 0.f ? 0u : (b & 0x80000000u) | 511u << 22 | (A != A ? 1u : 0u);
  return (b & 0x80000000u) | (((uint32_t)(max(-252, min(e + (int)(b >> 23 & 255u) - 127, 253)) + 256) << 22) + (((b & 0x7fffffu) + 1u) >> 1));
}
__device__ __forceinline__ Factors wide_factors(uint32_t code) {
  const int e = (int)(code >> 22 & 511u) - 256;
  const uint32_t sign = code & 0x80000000u;
  if (e == 255) return Factors(__uint_as_float(sign | 0x7f800000u | (code & 1u) << 22), 0);
  if (e == -256) return Factors(__uint_as_float(sign), 0);
  return Factors(__uint_as_float(sign | 0x3f800000u | (code & 0x3fffffu) << 1), e);
}

// ---- the chain through the cluster ----
// Per-CTA shared memory of the chain: parts (A0, A1, B0, B1 of a lane's two channels) and entering states per
// warp; mail, two steps of one part per CTA of the cluster.  A part whose A0 is a NaN has A0 and A1, and their
// exponents, in parts_m and parts_e, complete on a barrier of their own.  A second mail brings a tile's products
// outside fp32, in the steps that need them.
struct Chain {
  float4 *parts;    // [kScanWarps][32]
  float2 *parts_m;  // [kScanWarps][32]
  int *parts_e;     // [kScanWarps][32]
  float2 *enter;    // [kScanWarps][32]
  float4 *mail;     // [kMailSlots][cluster][32]
  int2 *wide_mail;  // [cluster][32], behind it
  uint64_t *parts_full, *products_full, *enter_full, *wide_full, *mail_full;  // the last: [kMailSlots]
  static constexpr int parts_bytes = kScanWarps * 32 * 16, parts_m_bytes = kScanWarps * 32 * 8, parts_e_bytes = kScanWarps * 32 * 4, enter_bytes = kScanWarps * 32 * 8;
  __host__ __device__ static constexpr int mail_bytes(int cluster) { return cluster * 32 * (kMailSlots * 16 + 8); }
  static constexpr int bars = 4 + kMailSlots;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_rank(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ void post16(uint32_t addr, float4 v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void post8(uint32_t addr, int2 v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(bar)
               : "memory");
}
// In the place of A where a sequence begins in the tile, so that its end state is B whatever enters
// (arithmetic never gives this NaN: its own has the sign bit clear).
constexpr uint32_t kCut = 0xffffffffu;

// A whole warp's wait on one of the CTA's barriers: bounded, one answer for all lanes.  False once this wait, or any other of the CTA, ran out: the
// calling role then stops (its outputs are undefined from there on); the other CTAs of the cluster stop
// likewise, for want of this one's mail.
// SHORT: the tries in a loop that is not unrolled.  Which is faster goes by the registers that a kernel gets (96, with a
// few spills): unrolled by the compiler and not, forward with log gates (65536 x 4096) 268 and 266 us, with sigmoid
// gates (64 packed requests) 210 and 217, backward from codes (65536 x 4096) 443 and 432.
template <bool SHORT>
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity, volatile int *gave_up, uint32_t *status, uint64_t limit_ns) {
  // sleeping tries first: the bounded wait begins with a read of the global timer, which takes longer
  // than most waits here (8 x 4096 x 2048 backward: 235 us with it alone, 150 us so)
  if constexpr (SHORT) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (__all_sync(0xffffffffu, sm100::mbar_try_sleep(bar, parity, 1000u))) return true;
  } else {
    for (int i = 0; i < 64; ++i)
      if (__all_sync(0xffffffffu, sm100::mbar_try_sleep(bar, parity, 1000u))) return true;
  }
  if (__all_sync(0xffffffffu, sm100::mbar_wait_or_abort(bar, parity, gave_up, limit_ns))) return true;
  set_status(status, GDP_DEV_ERR_TIMEOUT);
  return false;
}
// The loading warp, stopped before step n after a failed wait: its copies in flight (stages whose last use began before n).
template <int STAGES>
__device__ __forceinline__ void drain_loads(uint64_t *full, int n, bool words) {
  if (words) sm100::cp_async_wait_all();
  for (int i = n > STAGES ? n - STAGES : 0; i < n; ++i) (void)sm100::mbar_wait(&full[i % STAGES], (i / STAGES) & 1);
}
// Leaves the cluster: no CTA exits while another may still post to it.  After a failed wait posts may be
// under way that nobody waited for: they take microseconds at most.
__device__ __forceinline__ void leave_cluster(volatile int *gave_up) {
  __syncwarp();
  cluster_sync();
  if (*gave_up) {
    const uint64_t t0 = sm100::globaltimer_ns();
    while (sm100::globaltimer_ns() - t0 < 100000ull) __nanosleep(1000);
  }
}

// The largest decay of a lane's run, from the gates as they are stored, compared as integers (a NaN is on top); a
// sigmoid's decays are below one.
template <typename TG, int GATE>
struct LargestGate {
  static constexpr bool kWord = sizeof(TG) == 2;  // two channels in a word
  static constexpr bool kHalf = std::is_same<TG, __half>::value;
  // decays of 2^(1/16) and of 2^7: log gates of 0.0433 and 4.8125
  static constexpr int kRise = GATE == GDP_GATE_LOG ? (!kWord ? 0x3d317217 : kHalf ? 0x298b : 0x3d31) : (!kWord ? 0x3f85aac3 : kHalf ? 0x3c2d : 0x3f85);
  static constexpr int kSteep = GATE == GDP_GATE_LOG ? (!kWord ? 0x409a0000 : kHalf ? 0x44d0 : 0x409a) : (!kWord ? 0x43000000 : kHalf ? 0x5800 : 0x4300);
  static constexpr int kMask = GATE == GDP_GATE_LOG ? -1 : kWord ? 0x7fff7fff : 0x7fffffff;
  int x = kWord ? (int)0x80008000u : INT_MIN, y = INT_MIN;
  __device__ __forceinline__ void see(typename Packed<TG>::type v) {
    if constexpr (GATE != GDP_GATE_SIGMOID) {
      if constexpr (kWord) {
        asm("max.s16x2 %0, %0, %1;" : "+r"(x) : "r"((int)v & kMask));
      } else {
        x = max(x, __float_as_int(v.x) & kMask);
        y = max(y, __float_as_int(v.y) & kMask);
      }
    }
  }
  __device__ __forceinline__ bool above(int limit) const {
    if constexpr (GATE == GDP_GATE_SIGMOID) return false;
    else if constexpr (kWord) return max((int)(short)(x & 0xffff), x >> 16) > limit;
    else return max(x, y) > limit;
  }
  __device__ __forceinline__ bool rises() const { return above(kRise); }
  // The plain product holds all the same: up to 15 decays of 2^7 cannot bring back what a part of it had lost.
  __device__ __forceinline__ bool holds(float2 A) const {
    return !above(kSteep) && fminf(fabsf(A.x), fabsf(A.y)) >= 0x1p-15f && fmaxf(fabsf(A.x), fabsf(A.y)) <= 0x1p15f;
  }
};
// The products of S decays of a lane that is not safe, read again from the tile (out of line: few tiles come here).
template <typename TG, int GATE, bool RAW, int S>
__device__ __noinline__ void write_products(float2 *m, int *e, const unsigned char *gs, int row, int lane, RowSource src, int64_t t0, int64_t c0) {
  WideProduct x{1.f, 0}, y{1.f, 0};
#pragma unroll 1
  for (int i = 0; i < S; ++i) {
    float2 f;
    const float2 a = gate_decay<GATE>(gate_kept<GATE>(unpack<TG>(read_packed<TG, RAW>(gs, row + i, lane, RAW ? raw_offset<TG>(src, t0 + i, c0) : 0))), &f);
    x.times(a.x, 0);
    y.times(a.y, 0);
  }
  x.settle();
  y.settle();
  *m = make_float2(x.m, y.m);
  *e = pack_exponents(x.e, y.e);
}
// A computing warp, after its first run: writes its part, and says whether the lane's products have to follow (see
// write_products).  `cut`: a sequence begins among the tokens, A is one and is not used.
template <typename TG, int GATE>
__device__ __forceinline__ bool write_part(const Chain &ch, int at, float2 A, float2 B, const LargestGate<TG, GATE> &largest, bool cut) {
  const bool unsafe = !cut && (largest.rises() || !(fabsf(A.x) >= kSafe && fabsf(A.y) >= kSafe));
  ch.parts[at] = make_float4(unsafe ? __uint_as_float(0x7fffffffu) : A.x, A.y, B.x, B.y);
  return unsafe;
}
// A part, its exponents brought in.
__device__ __forceinline__ float4 read_part(const Chain &ch, int at, int &e) {
  float4 q = ch.parts[at];
  e = 0;
  if (q.x != q.x) {
    const float2 m = ch.parts_m[at];
    q.x = m.x;
    q.y = m.y;
    e = ch.parts_e[at];
  }
  return q;
}

// The cluster's tiles in order of time from the state h that enters the step, by plain products: the states that enter
// this CTA's tile and the next step, and whether those hold for this lane (every CTA finds the same).
struct StepStates {
  float2 enter, next;
  bool holds;
};
__device__ __forceinline__ StepStates plain_states(const float4 *mail, int cluster, int rank, int lane, float2 h) {
  float2 e = h;
  float least = kMost, most = 0.f, state = 0.f;
  for (int k0 = 0; k0 < cluster; k0 += 4) {
    float4 t[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k0 + u < cluster) t[u] = mail[(k0 + u) * 32 + lane];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (k0 + u >= cluster) break;
      if (k0 + u == rank) e = h;
      least = fminf(least, fminf(fabsf(t[u].x), fabsf(t[u].y)));  // (a cut tile has a NaN and a one)
      most = fmaxf(most, fmaxf(fabsf(t[u].x), fabsf(t[u].y)));
      state = fmaxf(state, fmaxf(fabsf(h.x), fabsf(h.y)));
      h = __float_as_uint(t[u].x) == kCut ? make_float2(t[u].z, t[u].w) : make_float2(fmaf(t[u].x, h.x, t[u].z), fmaf(t[u].y, h.y, t[u].w));
    }
  }
  return StepStates{e, h, most <= kMost && (least >= kSafe || state <= kLargeState)};
}

// The entering states are written; the slot's next mail may come (of step n + 2).
__device__ __forceinline__ void finish_step(const Chain &ch, int slot, uint32_t bytes, int lane) {
  __syncwarp();
  if (lane == 0) {
    sm100::mbar_arrive(ch.enter_full);
    sm100::mbar_arrive_expect_tx(&ch.mail_full[slot], bytes);
  }
}

// The chaining warp's step where plain products do not hold, out of line: before this CTA's mail is posted, when a part
// of its tile is not plain, or after (`posted`), when the cluster's mail shows that products outside fp32 matter.  Those
// come in a second mail, posted once the first has come, so that every CTA has read the step before's.  Costs 2.5 us a
// step (65536 x 4096 bf16 with log gates in -0.05 .. 0.05, all of whose steps come here: 578 against 265 us).
struct WideStep {
  float2 h;
  uint32_t phase;  // of the second mail
  bool ok;         // no wait ran out
};
static __device__ __noinline__ WideStep wide_step(Chain ch, int cluster, uint32_t *status, uint64_t limit_ns, uint32_t fresh, int n, int lane, float2 h, bool posted,
                                                  uint32_t phase, volatile int *gave_up) {
  const int rank = (int)cluster_rank(), slot = n % kMailSlots;
  if (!ring_wait<false>(ch.products_full, n & 1, gave_up, status, limit_ns)) return WideStep{h, phase, false};
  WideProduct x{1.f, 0}, y{1.f, 0};
  float2 B = make_float2(0.f, 0.f), A = both(1.f);  // A: as chain_steps has it
#pragma unroll 2
  for (int w = 0; w < kScanWarps; ++w) {
    int e;
    const float4 raw = ch.parts[w * 32 + lane], q = read_part(ch, w * 32 + lane, e);
    A = make_float2(A.x * raw.x, A.y * raw.y);
    x.times(q.x, low_exponent(e));
    y.times(q.y, high_exponent(e));
    B = w == 0 || (fresh >> w & 1u) ? make_float2(q.z, q.w)
                                    : make_float2(Factors(q.x, low_exponent(e)).apply(B.x, q.z), Factors(q.y, high_exponent(e)).apply(B.y, q.w));
  }
  x.settle();
  y.settle();
  if (!posted) {
    auto plain = [](WideProduct v) { return v.e == 0 ? v.m : v.e < 0 ? 0.f : __uint_as_float(0x7f800000u); };
    if (A.x != A.x) A = make_float2(plain(x), plain(y));
    const float4 own = make_float4(fresh ? __uint_as_float(kCut) : A.x, fresh ? 1.f : A.y, B.x, B.y);
    const uint32_t to = sm100::smem_u32(ch.mail + (slot * cluster + rank) * 32 + lane), full = sm100::smem_u32(&ch.mail_full[slot]);
    for (int k = 0; k < cluster; ++k) post16(in_rank(to, k), own, in_rank(full, k));
    if (!ring_wait<false>(&ch.mail_full[slot], (n / kMailSlots) & 1, gave_up, status, limit_ns)) return WideStep{h, phase, false};
  }
  const float4 *mail = ch.mail + slot * cluster * 32;
  const StepStates plain = plain_states(mail, cluster, rank, lane, h);
  float2 e = plain.enter, next = plain.next;
  if (!__all_sync(0xffffffffu, plain.holds)) {
    auto suspect = [](float v) { return fabsf(v) < kSafe || fabsf(v) > kMost; };
    uint32_t which = 0;  // tiles that send a second mail
    for (int k = 0; k < cluster; ++k) {
      const float4 t = mail[k * 32 + lane];
      which |= (__any_sync(0xffffffffu, __float_as_uint(t.x) != kCut && (suspect(t.x) || suspect(t.y))) ? 1u : 0u) << k;
    }
    if (which >> rank & 1u) {
      const uint32_t to = sm100::smem_u32(ch.wide_mail + rank * 32 + lane), full = sm100::smem_u32(ch.wide_full);
      const int2 codes = make_int2((int)wide_code(x.m, x.e), (int)wide_code(y.m, y.e));
      for (int k = 0; k < cluster; ++k) post8(in_rank(to, k), codes, in_rank(full, k));
    }
    if (lane == 0) sm100::mbar_arrive_expect_tx(ch.wide_full, (uint32_t)__popc(which) * 256u);
    if (!ring_wait<false>(ch.wide_full, phase, gave_up, status, limit_ns)) return WideStep{h, phase, false};
    phase ^= 1u;
    next = h;
    for (int k = 0; k < cluster; ++k) {
      const float4 t = mail[k * 32 + lane];
      if (k == rank) e = next;
      if (__float_as_uint(t.x) == kCut) {
        next = make_float2(t.z, t.w);
      } else {
        const int2 codes = which >> k & 1u ? ch.wide_mail[k * 32 + lane] : make_int2(0, 0);
        auto through = [&](float A, int code, float h, float add) {
          const bool wide = fabsf(A) > kMost || (fabsf(A) < kSafe && fabsf(h) > kLargeState);
          return wide ? wide_factors((uint32_t)code).apply(h, add) : fmaf(A, h, add);
        };
        next = make_float2(through(t.x, codes.x, next.x, t.z), through(t.y, codes.y, next.y, t.w));
      }
    }
  }
#pragma unroll 2
  for (int w = 0; w < kScanWarps; ++w) {
    int qe;
    const float4 q = read_part(ch, w * 32 + lane, qe);
    ch.enter[w * 32 + lane] = e;
    e = (fresh >> w & 1u) ? make_float2(q.z, q.w)
                          : make_float2(Factors(q.x, low_exponent(qe)).apply(e.x, q.z), Factors(q.y, high_exponent(qe)).apply(e.y, q.w));
  }
  finish_step(ch, slot, (uint32_t)cluster * 512u, lane);
  return WideStep{next, phase, true};
}

// The chaining warp.  Mail slots: a CTA posts step n + 2 only after it has read the mail of step n + 1,
// which holds this CTA's post of n + 1, which this warp sent after it had read step n: two suffice.
// parts: a warp writes tile n + 1's after its entering state of tile n, which was formed from tile n's.
// (Backward, the tiles and the tokens in them go back in time, and the ends of sequences cut the chain.)
template <int S, int META, bool SHORT>
__device__ __forceinline__ void chain_steps(const ScanShape &p, const Chain &ch, const TileMeta<S> *metas, int steps, int lane,
                                            volatile int *gave_up) {
  const uint32_t rank = cluster_rank(), bytes = (uint32_t)p.cluster * 512u;
  if (lane == 0)
    for (int i = 0; i < kMailSlots; ++i) sm100::mbar_arrive_expect_tx(&ch.mail_full[i], bytes);
  float2 h = make_float2(0.f, 0.f);  // the state entering the step
  uint32_t phase = 0;
  for (int n = 0; n < steps; ++n) {
    if (!ring_wait<SHORT>(ch.parts_full, n & 1, gave_up, p.status, p.limit_ns)) return;
    const uint32_t fresh = metas[n % META].fresh;
    const int slot = n % kMailSlots;
    float4 q[kScanWarps];
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) q[w] = ch.parts[w * 32 + lane];
    float4 own = q[0];
#pragma unroll
    for (int w = 1; w < kScanWarps; ++w) {
      const bool f = fresh >> w & 1u;
      own = make_float4(own.x * q[w].x, own.y * q[w].y, f ? q[w].z : fmaf(q[w].x, own.z, q[w].z), f ? q[w].w : fmaf(q[w].y, own.w, q[w].w));
    }
    auto wide = [&](bool posted) {
      const WideStep step = wide_step(ch, p.cluster, p.status, p.limit_ns, fresh, n, lane, h, posted, phase, gave_up);
      h = step.h;
      phase = step.phase;
      return step.ok;
    };
    if (__builtin_expect(__any_sync(0xffffffffu, own.x != own.x), 0)) {  // some part is not plain
      if (!wide(false)) return;
      continue;
    }
    if (fresh) {
      own.x = __uint_as_float(kCut);
      own.y = 1.f;
    }
    const uint32_t to = sm100::smem_u32(ch.mail + (slot * p.cluster + (int)rank) * 32 + lane);
    const uint32_t bar = sm100::smem_u32(&ch.mail_full[slot]);
    if (!(p.withhold && n == 0 && rank == 0)) {
#pragma unroll 4
      for (int k = 0; k < p.cluster; ++k) post16(in_rank(to, k), own, in_rank(bar, k));
    }
    if (!ring_wait<SHORT>(&ch.mail_full[slot], (n / kMailSlots) & 1, gave_up, p.status, p.limit_ns)) return;
    const StepStates states = plain_states(ch.mail + slot * p.cluster * 32, p.cluster, (int)rank, lane, h);
    if (__builtin_expect(!__all_sync(0xffffffffu, states.holds), 0)) {
      if (!wide(true)) return;
      continue;
    }
    h = states.next;
    float2 e = states.enter;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) {
      ch.enter[w * 32 + lane] = e;
      e = (fresh >> w & 1u) ? make_float2(q[w].z, q[w].w) : make_float2(fmaf(q[w].x, e.x, q[w].z), fmaf(q[w].y, e.y, q[w].w));
    }
    finish_step(ch, slot, bytes, lane);
  }
}

struct RecFwd {
  ScanShape s;
  RowSource x, g;
  void *h;
  const float *from;  // state rows read (initial state or cache)
  float *to;          // state rows written (final state or cache)
  int pair_out;       // two channels of h can be stored at once
  int vec_out;        // h can be stored by TMA
};
struct RecBwd {
  ScanShape s;
  RowSource g, x, h, dout;
  RowSource codes;     // int8
  const float *scales;
  int64_t group;       // channels of a checkpoint row
  int64_t blocks;      // scales of a checkpoint row
  const float *init, *dfin;
  void *dx, *dg;
  float *dinit;
  int pair_dx, pair_dg;  // two channels can be stored at once
  int vec_out;           // dx and dg can be stored by TMA
};

// Fills s.rows, s.slices and s.cluster and launches (instantiated in gdp_rec_*.cu).
template <typename TX, typename TG>
cudaError_t launch_rec_fwd(RecFwd &p, int gate, cudaStream_t stream);
template <typename TX, typename TG>
cudaError_t launch_rec_bwd(RecBwd &p, int gate, cudaStream_t stream);
// CTAs per slice: a power of two that fills every SM with `per_sm` (9 CTAs per cluster instead of 8 took
// 458 us instead of 288 us at C = 2048), at most one per tile in time.  Clusters of 16 start slowly and pay
// only for few channels and many tiles (us with 8 / 16 CTAs: 65536 x 512 106 / 77, 65536 x 1024 128 / 139,
// 8192 x 512 16.5 / 12.6, 8192 x 1024 19.0 / 22.9, 1421 x 1024 8.1 / 13.3, all when this was chosen).
inline int cluster_size(int slices, int rows, int sms, int per_sm) {
  int k = sms * per_sm / (slices > 0 ? slices : 1);
  if (k > rows) k = rows;
  const int most = slices <= 8 && rows > 24 ? 16 : 8;
  int pow = 1;
  while (2 * pow <= k && pow < most) pow *= 2;
  return pow;
}
// Launches slices x cluster CTAs in clusters.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kern)(Params...), int slices, int cluster, int smem, cudaStream_t stream, Args &&...args) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && cluster > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(slices * cluster));
  cfg.blockDim = dim3(kScanThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args &&>(args)...);
}
// SMs of the current device.
int sm_count();

}  // namespace layer

// TMA map of a row-major matrix of 1-, 2- or 4-byte elements, unswizzled boxes of box_cols x box_rows
// (gdp_tmap.cu; `map` points at a 64-byte aligned CUtensorMap).
cudaError_t tmap_matrix(void *map, const void *base, int64_t rows, int64_t cols, int64_t stride_bytes, int elem_bytes, int box_cols,
                        int box_rows);
}  // namespace gdp
