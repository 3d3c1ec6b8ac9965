// gdp_rec_bf16.cu -- the recurrence's scans over bf16 inputs.
#include "gdp_rec_fwd_body.cuh"

cudaError_t gdp::layer::launch_rec_fwd_bf16(RecFwd &p, int g_f32, int gate, cudaStream_t stream) {
  return g_f32 ? run_fwd_gate<__nv_bfloat16, float>(p, gate, stream) : run_fwd_gate<__nv_bfloat16, __nv_bfloat16>(p, gate, stream);
}
