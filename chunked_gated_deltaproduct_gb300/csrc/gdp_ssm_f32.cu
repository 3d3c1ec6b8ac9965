// gdp_ssm_f32.cu -- the selective state space scan over f32 rows, forward.
#include "gdp_ssm_fwd_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_ssm_fwd<float>(const SsmProblem &, cudaStream_t);
template cudaError_t launch_ssm_step<float>(const SsmProblem &, cudaStream_t);
}  // namespace layer
}  // namespace gdp
