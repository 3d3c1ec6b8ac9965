// gdp_rec_f16.cu -- the recurrence's scans over f16 inputs.
#include "gdp_rec_fwd_body.cuh"

cudaError_t gdp::layer::launch_rec_fwd_f16(RecFwd &p, int g_f32, int gate, cudaStream_t stream) {
  return g_f32 ? run_fwd_gate<__half, float>(p, gate, stream) : run_fwd_gate<__half, __half>(p, gate, stream);
}
