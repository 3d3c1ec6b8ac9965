// gdp_rec_f32.cu -- the recurrence's scans over f32 inputs.
#include "gdp_rec_fwd_body.cuh"

cudaError_t gdp::layer::launch_rec_fwd_f32(RecFwd &p, int, int gate, cudaStream_t stream) {
  return run_fwd_gate<float, float>(p, gate, stream);
}
