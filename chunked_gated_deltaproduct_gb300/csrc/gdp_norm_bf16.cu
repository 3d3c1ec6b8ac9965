// gdp_norm_bf16.cu -- the grouped norm's kernels over bf16 tensors.
#include "gdp_norm_body.cuh"

template cudaError_t gdp::layer::launch_norm_fwd<__nv_bfloat16>(const NormProblem &, const NormPlan &, cudaStream_t);
template cudaError_t gdp::layer::launch_norm_bwd<__nv_bfloat16>(const NormProblem &, const NormPlan &, cudaStream_t);
