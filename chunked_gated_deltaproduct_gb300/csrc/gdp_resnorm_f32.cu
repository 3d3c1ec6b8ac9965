// gdp_resnorm_f32.cu -- the residual norm over f32 blocks.
#include "gdp_resnorm_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_res_fwd<float>(ResProblem &, int, cudaStream_t);
template cudaError_t launch_res_bwd<float>(ResProblem &, int, int64_t, cudaStream_t);
}  // namespace layer
}  // namespace gdp
