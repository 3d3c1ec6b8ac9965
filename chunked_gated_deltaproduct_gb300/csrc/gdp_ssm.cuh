// gdp_ssm.cuh -- the selective state space scan's problem and launchers.
#pragma once

#include <cmath>

#include "gdp_block.cuh"

namespace gdp {
namespace layer {

struct SsmProblem {
  const void *x, *dt, *z, *B, *Cm;
  int64_t x_st, dt_st, z_st, B_st, B_sg, C_st, C_sg;
  const float *A, *D, *bias;
  void *y;
  Packed p;
  int64_t C, S, G;
  int64_t per;         // channels of a group
  int tiles;           // CTAs that share a group's channels
  StateModes s;
  float *chunks;       // states entering every chunk, written by the forward and read by the backward pass
  int dt_f32, softplus, zero_pad;
  int sms;             // of the device
  int fast_rows;       // x, dt and z can be copied by 16 bytes from every CTA's first channel on
  int fast_vectors;    // B and C likewise
  int quad_vectors;    // A, B and C can be read by four states
  int pair_out;        // outputs can be written by two channels
  int quad_states;     // four states at a time: S a multiple of four, every state buffer on 16 bytes
  // Pieces: where whole sequences leave SMs idle, pieces of `piece` tokens (0: whole sequences) run side by side, first
  // from zero for the states they reach, which are then joined to the states entering them.
  int64_t piece, pieces;  // tokens; rows of pieces (or sequences)
  int ranked;             // whole sequences, the longest first
  float *enter, *spans;   // [pieces][C][S] and [pieces][C]
  // backward
  const void *dy;
  int64_t dy_st;
  const float *dfin;
  void *dx, *ddt, *dz, *dB, *dC;
  float *dinit;
  float *over_rows;      // [workers][ssm_sum_cols]: sums over a worker's rows for dA, dD, ddt_bias
  float *over_channels;  // [G tiles][T][2 padded S]: a CTA's channels' sums for dB and dC
  int64_t workers;       // CTAs that share the sequences
};

constexpr int kSsmThreads = 128;
constexpr int kSsmChunk = GDP_SCAN_CHUNK;

// Lanes that share a channel, four states each.
inline int ssm_lanes(int64_t S) { return S <= 16 ? 4 : S <= 32 ? 8 : 16; }
inline int64_t ssm_tiles(int64_t per, int64_t S) { return (per * ssm_lanes(S) + kSsmThreads - 1) / kSsmThreads; }
// Sequences that are ranked by length: where there are more CTAs than are resident at once, the longest come first, so that
// none of them is what the last SMs wait for (64 packed requests of 16 to 8192 tokens x 2048, forward: 1254 us in
// their own order, 1011 so).  Every CTA ranks them, which takes about as long as N / 3 tokens: where the mean sequence is
// shorter than N they run in their own order (200 of a token x 2048: 83 us, ranked 230; 64 of 30: 61 and 65; 26 of 30: 43 and 41).
constexpr int kSsmRanked = 256;
inline bool ssm_ranked(int64_t T, int64_t N, int64_t tiles, int sms) { return N > 1 && N <= kSsmRanked && T >= N * N && N * tiles > 2 * sms; }
// Workers of the backward pass: as many as give every SM 16 CTAs, and no more than there are sequences.
inline int64_t ssm_workers(int64_t N, int64_t tiles, int sms) {
  int64_t n = (16 * (int64_t)sms + tiles - 1) / tiles;
  if (n > N) n = N;
  return n < 1 ? 1 : n;
}

// Tokens of a piece, 0 for whole sequences, from the shape alone (the lengths are the device's).  Pieces add a pass and two
// launches, and use the SMs that whole sequences leave idle: as many pieces as are resident at once (`per_sm` CTAs on an
// SM), unless they became long; then three waves or more of shorter ones.  Joining takes the pieces of a sequence one by one, 0.18 us
// each where a piece's token takes 0.06 (backward 0.24): the square root.
// Measured on the device, whole sequences against pieces, us (bf16, S = 16):
//   forward   1 x 256 x 256 13.1 to 11.9, 1 x 256 x 1024 13.4 to 14.4, 1 x 512 x 2048 22 to 24, 1 x 1000 x 1024 43 to 24,
//             1 x 4096 x 512 161 to 36, 1 x 65536 x 1024 2533 to 633; 100, 257, 64 and 1000 x 1024 43 to 31
//   backward  1 x 96 x 256 27 to 23, 1 x 256 x 256 57 to 24, 1 x 512 x 2048 118 to 68, 1 x 1000 x 4096 223 to 194, two of
//             100 x 512 32 to 27
// Equal sequences that fill more than the SMs' half lose by it (forward, 4 x 4096 x 1024 162 to 186), ragged ones win.
// Shorter pieces than fill the SMs once cost a second wave (backward, 1 x 4096 x 512: 224 tokens 81 us, 192 127).
inline int64_t ssm_piece(int64_t T, int64_t N, int64_t tiles, int sms, int per_sm) {
  const bool back = per_sm == 2;
  const int64_t whole = N * tiles, slots = (int64_t)per_sm * sms;
  if (T < 96 * N || (N > 1 ? 2 * whole >= 3 * sms || (!back && T < 256 * N) : back ? whole > sms : 10 * whole >= 6 * sms)) return 0;
  int64_t n = (T * tiles + slots - 1) / slots;
  if (n > 512) n = (T * tiles + 6 * sms - 1) / (6 * sms);
  const int64_t least = (int64_t)std::sqrt((back ? 1. : 2.) * (double)T);
  if (n < least) n = least;
  n = (n + 31) / 32 * 32;
  if (n < 32) n = 32;
  // (forward, one sequence: a launch's time is that of 150 tokens, a piece's token of 2.1 whole ones, a full SM of 200)
  if (!back && N == 1 && 150 + 2 * n + 200 * T * tiles / (n * slots) >= T) return 0;
  return n;
}
constexpr int kSsmForward = 3, kSsmBackward = 2;  // CTAs on an SM

// Columns of the backward pass's sums over rows: C S, C and C, and up to a multiple of 16 bytes.
__host__ __device__ inline int64_t ssm_sum_cols(int64_t C, int64_t S) { return (C * (S + 2) + 3) / 4 * 4; }

template <typename T>
cudaError_t launch_ssm_fwd(const SsmProblem &p, cudaStream_t stream);
template <typename T>
cudaError_t launch_ssm_step(const SsmProblem &p, cudaStream_t stream);
template <typename T>
cudaError_t launch_ssm_bwd(const SsmProblem &p, cudaStream_t stream);

}  // namespace layer
}  // namespace gdp
