// gdp_norm_f32.cu -- the grouped norm's kernels over f32 tensors.
#include "gdp_norm_body.cuh"

template cudaError_t gdp::layer::launch_norm_fwd<float>(const NormProblem &, const NormPlan &, cudaStream_t);
template cudaError_t gdp::layer::launch_norm_bwd<float>(const NormProblem &, const NormPlan &, cudaStream_t);
