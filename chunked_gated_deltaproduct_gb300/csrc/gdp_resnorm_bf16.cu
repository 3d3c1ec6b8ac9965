// gdp_resnorm_bf16.cu -- the residual norm over bf16 blocks.
#include "gdp_resnorm_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_res_fwd<__nv_bfloat16>(ResProblem &, int, cudaStream_t);
template cudaError_t launch_res_bwd<__nv_bfloat16>(ResProblem &, int, int64_t, cudaStream_t);
}  // namespace layer
}  // namespace gdp
