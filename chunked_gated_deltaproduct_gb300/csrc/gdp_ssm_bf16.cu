// gdp_ssm_bf16.cu -- the selective state space scan over bf16 rows, forward.
#include "gdp_ssm_fwd_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_ssm_fwd<__nv_bfloat16>(const SsmProblem &, cudaStream_t);
template cudaError_t launch_ssm_step<__nv_bfloat16>(const SsmProblem &, cudaStream_t);
}  // namespace layer
}  // namespace gdp
