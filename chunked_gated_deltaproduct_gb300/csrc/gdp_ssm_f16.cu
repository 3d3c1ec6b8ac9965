// gdp_ssm_f16.cu -- the selective state space scan over f16 rows, forward.
#include "gdp_ssm_fwd_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_ssm_fwd<__half>(const SsmProblem &, cudaStream_t);
template cudaError_t launch_ssm_step<__half>(const SsmProblem &, cudaStream_t);
}  // namespace layer
}  // namespace gdp
