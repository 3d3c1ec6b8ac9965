// gdp_conv.cuh -- the short causal convolution's problem and launchers.
#pragma once

#include "gdp_block.cuh"

namespace gdp {
namespace layer {

struct ConvProblem {
  const void *x;
  int64_t x_st;
  const float *w, *b;
  void *y;
  Packed p;
  int64_t C;
  StateModes s;
  int act, zero_pad;
  int quad_taps;   // weight on a 16-byte boundary
  // backward
  const void *dy;
  int64_t dy_st;
  const void *dfin;
  void *dx, *dinit;
  float *partial;  // [parts][W + 1][C]
  // plan
  int64_t run, runs;  // forward: rows of a thread; CTAs over rows (both passes)
  int64_t parts, part_rows;
};

constexpr int kConvThreads = 128;
// A CTA is `x` vectors of channels by `y` runs of rows: rows as wide as can be without more than an eighth of the threads idle.
inline dim3 conv_block(int64_t vecs) {
  int x = 1;
  while (x < 32 && x < vecs) x *= 2;
  while (x >= 32 && x < kConvThreads && (vecs + 2 * x - 1) / (2 * x) * (2 * x) * 8 <= vecs * 9) x *= 2;
  return dim3(x, kConvThreads / x);
}

template <typename T>
cudaError_t launch_conv_fwd(ConvProblem &p, int width, int vec, bool states, cudaStream_t stream);
template <typename T>
cudaError_t launch_conv_states(const ConvProblem &p, int width, cudaStream_t stream);
template <typename T>
cudaError_t launch_conv_step(const ConvProblem &p, int width, cudaStream_t stream);
template <typename T>
cudaError_t launch_conv_bwd(ConvProblem &p, int width, int vec, cudaStream_t stream);

// Parts of the rows whose weight gradients are summed apart, by the vectors of channels in a row: as many CTAs as are
// resident at once (four per SM), of eight rows or more a thread (of 64 or more: 900 x 1280 21 us, eight 13; 5000 x 2048 31 and
// 27; from 20000 x 2048 on the SMs are full either way).
inline int64_t conv_parts(int64_t T, int64_t vecs, int sms) {
  const int64_t y = conv_block(vecs).y, x = conv_block(vecs).x;
  const int64_t across = (vecs + x - 1) / x;
  int64_t ctas = sms * 4 / across;
  const int64_t most = (T + 8 * y - 1) / (8 * y);
  if (ctas > most) ctas = most;
  if (ctas < 1) ctas = 1;
  return ctas * y;
}

}  // namespace layer
}  // namespace gdp
