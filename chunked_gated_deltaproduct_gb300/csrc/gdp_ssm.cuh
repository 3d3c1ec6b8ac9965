// gdp_ssm.cuh -- the selective state space scan's problem and launchers.
#pragma once

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
// Sequences that can be ranked by length: where there are more CTAs than are resident at once, the longest come first, so that
// none of them is what the last SMs wait for (64 packed requests of 16 to 8192 tokens x 2048, forward: 1254 us in
// their own order, 1011 so).
constexpr int kSsmRanked = 256;
inline bool ssm_ranked(int64_t N, int64_t tiles, int sms) { return N > 1 && N <= kSsmRanked && N * tiles > 2 * sms; }
// Workers of the backward pass: as many as give every SM 16 CTAs, and no more than there are sequences.
inline int64_t ssm_workers(int64_t N, int64_t tiles, int sms) {
  int64_t n = (16 * (int64_t)sms + tiles - 1) / tiles;
  if (n > N) n = N;
  return n < 1 ? 1 : n;
}

// Tokens of a piece, 0 for whole sequences, from the shape alone (the lengths are the device's).  A sequence alone
// takes 34 ns a token; pieces add a pass of 0.6 of the first one's time and about 13 us, and use the SMs that whole
// sequences leave idle.  Measured on the device, whole sequences against pieces (bf16, S = 16): 1 x 65536 x 1024 2533 to
// 697 us, 1 x 4096 x 512 161 to 43, 1 x 1000 x 1024 43 to 27, 2 x 4096 x 1024 162 to 120; equal sequences of half the SMs'
// CTAs or more lose (4 x 4096 x 1024 162 to 186), ragged ones win (100, 257, 64 and 1000 tokens x 1024: 43 to 27).
inline int64_t ssm_piece(int64_t T, int64_t N, int64_t tiles, int sms) {
  const int64_t whole = N * tiles;
  if (N == 1 ? T < 512 || 10 * whole >= 6 * sms : T < 256 * N || 2 * whole >= 3 * sms) return 0;
  int64_t n = (T * tiles + 6 * sms - 1) / (6 * sms);  // six CTAs per SM
  if (n < T / 192) n = T / 192;                       // (joining takes the pieces of a sequence one by one)
  n = (n + 31) / 32 * 32;
  return n < 128 ? 128 : n;
}

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
