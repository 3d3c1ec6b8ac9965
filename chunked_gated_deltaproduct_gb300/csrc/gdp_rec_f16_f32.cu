// gdp_rec_f16_f32.cu -- the recurrence's scans: f16 inputs, fp32 gates.
#include "gdp_rec_bwd_body.cuh"
#include "gdp_rec_fwd_body.cuh"

template cudaError_t gdp::layer::launch_rec_fwd<__half, float>(RecFwd &, int, cudaStream_t);
template cudaError_t gdp::layer::launch_rec_bwd<__half, float>(RecBwd &, int, cudaStream_t);
