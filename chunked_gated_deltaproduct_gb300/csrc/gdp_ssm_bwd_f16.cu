// gdp_ssm_bwd_f16.cu -- the selective state space scan over f16 rows, backward.
#include "gdp_ssm_bwd_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_ssm_bwd<__half>(const SsmProblem &, cudaStream_t);
}  // namespace layer
}  // namespace gdp
