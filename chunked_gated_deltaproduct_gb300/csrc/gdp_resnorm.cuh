// gdp_resnorm.cuh -- the residual norm's problem and launchers.
#pragma once

#include "gdp_block.cuh"

namespace gdp {
namespace layer {

struct ResProblem {
  const void *res, *block, *gate;
  int64_t res_st, block_st, gate_st;
  const float *w, *post, *scale;
  void *y, *r;
  int64_t T, C;
  float eps, inv_c;
  int act, res_f32;
  int quad_cols;  // weights on 16-byte boundaries
  int keep;       // backward: weights are held in shared memory
  int depth;      // rows that a thread has places for in shared memory
  // backward (res is the forward's residual_out)
  const void *dy, *dr;
  int64_t dy_st, dr_st;
  void *dres, *dblock, *dgate;
  float *partial;  // [parts][3][C]: sums for weight, post_weight, scale
};

constexpr int kRes = 8;         // channels of a thread
constexpr int kResMost = 8192;  // channels
// Threads of a row, eight channels each: a warp, or a whole CTA.
inline int res_threads(int64_t C) { return (int)((C + 255) / 256) * 32; }
inline int res_rows(int64_t C) { return C <= 256 ? 4 : 1; }  // rows of a CTA at a time
// CTAs of the backward pass (each adds up its rows' columns): 512 threads per SM are resident at its registers.
constexpr int kResResident = 512;
inline int64_t res_ctas(int64_t T, int64_t C, int sms) {
  const int threads = res_threads(C) * res_rows(C);
  int64_t n = (int64_t)sms * (threads < kResResident ? kResResident / threads : 1);
  const int64_t need = (T + res_rows(C) - 1) / res_rows(C);
  if (n > need) n = need;
  return n < 1 ? 1 : n;
}

template <typename T>
cudaError_t launch_res_fwd(ResProblem &p, int vec, cudaStream_t stream);
template <typename T>
cudaError_t launch_res_bwd(ResProblem &p, int vec, int64_t ctas, cudaStream_t stream);

}  // namespace layer
}  // namespace gdp
