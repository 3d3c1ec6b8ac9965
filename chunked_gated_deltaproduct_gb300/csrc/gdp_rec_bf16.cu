// gdp_rec_bf16.cu -- the recurrence's scans: bf16 inputs, bf16 gates.
#include "gdp_rec_bwd_body.cuh"
#include "gdp_rec_fwd_body.cuh"

template cudaError_t gdp::layer::launch_rec_fwd<__nv_bfloat16, __nv_bfloat16>(RecFwd &, int, cudaStream_t);
template cudaError_t gdp::layer::launch_rec_bwd<__nv_bfloat16, __nv_bfloat16>(RecBwd &, int, cudaStream_t);
