// gdp_rec_f32.cu -- the recurrence's scans: fp32 inputs and gates.
#include "gdp_rec_bwd_body.cuh"
#include "gdp_rec_fwd_body.cuh"

template cudaError_t gdp::layer::launch_rec_fwd<float, float>(RecFwd &, int, cudaStream_t);
template cudaError_t gdp::layer::launch_rec_bwd<float, float>(RecBwd &, int, cudaStream_t);
