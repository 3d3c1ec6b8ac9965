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
  int depth;      // rows that a thread has places for in shared memory
  // backward (res is the forward's residual_out)
  const void *dy, *dr;
  int64_t dy_st, dr_st;
  void *dres, *dblock, *dgate;
  float *partial;  // [parts][3][C]: sums for weight, post_weight, scale
};

constexpr int kRes = 8;         // channels of a thread
constexpr int kResMost = 8192;  // channels
// A row's CTAs in the backward pass: beyond 4096 channels a pair on two SMs, which exchange their sums (a CTA of 1024 threads
// has 64 registers a thread, which do not hold what it needs: 32768 x 8192 bf16, fp32 stream: 2692 us, a pair's 1554; 5120:
// 1654 and 1087).  The forward pass fits (32768 x 8192: 1044 us, a pair 1130).
inline int res_cluster(int64_t C) { return C > 4096 ? 2 : 1; }
// Threads of each of a row's CTAs, eight channels a thread: whole warps.
inline int res_threads(int64_t C, int ctas) { return (int)((C + 256 * ctas - 1) / (256 * ctas)) * 32; }
inline int res_rows(int64_t C) { return C <= 256 ? 4 : 1; }  // rows of a CTA at a time
// CTAs, or pairs of them, of the backward pass (each adds up its rows' columns): 512 threads per SM are resident at its registers.
constexpr int kResResident = 512;
inline int64_t res_parts(int64_t T, int64_t C, int sms) {
  const int threads = res_threads(C, res_cluster(C)) * res_rows(C);
  int64_t n = (int64_t)sms * (threads < kResResident ? kResResident / threads : 1) / res_cluster(C);
  const int64_t need = (T + res_rows(C) - 1) / res_rows(C);
  if (n > need) n = need;
  return n < 1 ? 1 : n;
}

template <typename T>
cudaError_t launch_res_fwd(ResProblem &p, int vec, cudaStream_t stream);
template <typename T>
cudaError_t launch_res_bwd(ResProblem &p, int vec, int64_t parts, cudaStream_t stream);

}  // namespace layer
}  // namespace gdp
