// gdp_norm_f16.cu -- the grouped norm's kernels over f16 tensors.
#include "gdp_norm_body.cuh"

template cudaError_t gdp::layer::launch_norm_fwd<__half>(const NormProblem &, const NormPlan &, cudaStream_t);
template cudaError_t gdp::layer::launch_norm_bwd<__half>(const NormProblem &, const NormPlan &, cudaStream_t);
