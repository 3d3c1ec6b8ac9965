// gdp_rec_f16.cu -- the recurrence's scans: f16 inputs, f16 gates.
#include "gdp_rec_bwd_body.cuh"
#include "gdp_rec_fwd_body.cuh"

template cudaError_t gdp::layer::launch_rec_fwd<__half, __half>(RecFwd &, int, cudaStream_t);
template cudaError_t gdp::layer::launch_rec_bwd<__half, __half>(RecBwd &, int, cudaStream_t);
