// gdp_resnorm_f16.cu -- the residual norm over f16 blocks.
#include "gdp_resnorm_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_res_fwd<__half>(ResProblem &, int, cudaStream_t);
template cudaError_t launch_res_bwd<__half>(ResProblem &, int, int64_t, cudaStream_t);
}  // namespace layer
}  // namespace gdp
