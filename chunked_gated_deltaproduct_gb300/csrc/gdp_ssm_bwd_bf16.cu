// gdp_ssm_bwd_bf16.cu -- the selective state space scan over bf16 rows, backward.
#include "gdp_ssm_bwd_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_ssm_bwd<__nv_bfloat16>(const SsmProblem &, cudaStream_t);
}  // namespace layer
}  // namespace gdp
