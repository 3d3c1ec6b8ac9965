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
  int64_t per, tiles;  // channels of a group; CTAs that share a group's channels
  StateModes s;
  float *chunks;       // states entering every chunk, written by the forward and read by the backward pass
  int dt_f32, softplus, zero_pad;
  int quad_states;     // four states at a time: S a multiple of four, every state buffer on 16 bytes
  // backward
  const void *dy;
  int64_t dy_st;
  const float *dfin;
  void *dx, *ddt, *dz, *dB, *dC;
  float *dinit;
  float *over_rows;      // [workers][C (S + 2)]: sums over a worker's rows for dA, dD, ddt_bias
  float *over_channels;  // [G tiles][T][2 padded S]: a CTA's channels' sums for dB and dC
  int64_t workers;       // CTAs that share the sequences
};

constexpr int kSsmThreads = 128;
constexpr int kSsmChunk = GDP_SCAN_CHUNK;

// Lanes that share a channel, four states each.
inline int ssm_lanes(int64_t S) { return S <= 16 ? 4 : S <= 32 ? 8 : 16; }
inline int64_t ssm_tiles(int64_t per, int64_t S) { return (per * ssm_lanes(S) + kSsmThreads - 1) / kSsmThreads; }
// Workers of the backward pass: as many as fill the SMs four times, and no more than there are sequences.
inline int64_t ssm_workers(int64_t N, int64_t tiles, int sms) {
  int64_t n = (4 * (int64_t)sms + tiles - 1) / tiles;
  if (n > N) n = N;
  return n < 1 ? 1 : n;
}

template <typename T>
cudaError_t launch_ssm_fwd(const SsmProblem &p, cudaStream_t stream);
template <typename T>
cudaError_t launch_ssm_step(const SsmProblem &p, cudaStream_t stream);
template <typename T>
cudaError_t launch_ssm_bwd(const SsmProblem &p, cudaStream_t stream);

}  // namespace layer
}  // namespace gdp
