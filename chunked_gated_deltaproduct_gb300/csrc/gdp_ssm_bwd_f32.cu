// gdp_ssm_bwd_f32.cu -- the selective state space scan over f32 rows, backward.
#include "gdp_ssm_bwd_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_ssm_bwd<float>(const SsmProblem &, cudaStream_t);
}  // namespace layer
}  // namespace gdp
