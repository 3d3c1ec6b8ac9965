// gdp_norm.cuh -- the grouped norm's problem, launch plan and launchers.
#pragma once

#include <type_traits>

#include "gdp_layer.cuh"
#include "gdp_sm100.cuh"

namespace gdp {
namespace layer {

struct NormProblem {
  const void *o, *z;
  int64_t o_st, o_sh, z_st, z_sh;
  const int8_t *o_codes_in, *z_codes_in;  // backward: read instead of o and z
  const float *o_scales_in, *z_scales_in;
  const float *w, *b;
  void *y;
  int8_t *o_codes, *z_codes;
  float *o_scales, *z_scales;
  const void *dy;
  int64_t dy_st, dy_sh;
  void *d_o, *d_z;
  float *dw, *db, *partial;
  int64_t T, H, D;
  int64_t heads, groups, parts;  // see NormPlan
  float eps, inv_d;
  int center, per_head, act;
  int vec_cols;  // weight and bias rows start on 16-byte boundaries
};

// Threads of a CTA: groups of L lanes (L > 0), or one group (L = 0: up to 512 threads).
template <int L>
constexpr int kNormThreads = L > 0 ? 256 : 512;

// Resident CTAs of 256 threads per SM: what the registers allow with next to no spills (forward 80, backward
// 128 registers, 8 to 28 bytes spilled; four and three: 915 us and 1240 us for the training step of 65536 x 32 x 128, so:
// 784 us).
constexpr int kNormFwdCtas = 3, kNormBwdCtas = 2;
// How a call runs: groups of `lanes` threads (0: a CTA of `threads`), sixteen channels each.
// The groups number grid * (groups per CTA), a multiple of `heads`; group i keeps head i % heads (none
// when that is H or more), and there are `parts` column sums to add up.
struct NormPlan {
  int vec, lanes, threads;
  int64_t grid, heads, groups, parts;
};

inline NormPlan norm_plan(int64_t T, int64_t H, int64_t D, int per_head, int vec, int sms, int per_sm) {
  NormPlan n{};
  n.vec = vec;
  n.threads = 256;
  if (D <= 64 && vec) n.lanes = 4;
  else if (D <= 128) n.lanes = 8;
  else if (D <= 256 && vec) n.lanes = 16;
  else if (D <= 512) n.lanes = 32;
  else n.threads = (int)((D + 511) / 512 * 32);
  const int64_t per_cta = n.lanes ? n.threads / n.lanes : 1;
  // CTAs must come in multiples of m for every group to keep its head; where that is too coarse, heads
  // are rounded up to whole CTAs and the last groups have none
  int64_t a = H, b = per_cta;
  while (b) {
    const int64_t c = a % b;
    a = b;
    b = c;
  }
  int64_t m = H / a;
  n.heads = H;
  if (m > 32) {
    n.heads = (H + per_cta - 1) / per_cta * per_cta;
    m = n.heads / per_cta;
  }
  // CTAs of 256 threads: a few per SM; smaller ones: as many threads
  const int64_t resident = (int64_t)sms * (n.threads >= 256 ? per_sm : per_sm * 256 / n.threads);
  const int64_t need = (T * n.heads + per_cta - 1) / per_cta;
  n.grid = (need + m - 1) / m * m;
  if (n.grid > resident) n.grid = resident / m * m;
  if (n.grid < m) n.grid = m;
  n.groups = n.grid * per_cta;
  n.parts = per_head ? n.groups / n.heads : n.grid;
  return n;
}

template <typename T>
cudaError_t launch_norm_fwd(const NormProblem &p, const NormPlan &n, cudaStream_t stream);
template <typename T>
cudaError_t launch_norm_bwd(const NormProblem &p, const NormPlan &n, cudaStream_t stream);

int sm_count();  // of the current device (gdp_recurrence.cu)

}  // namespace layer
}  // namespace gdp
