// gdp_conv_bf16.cu -- the short causal convolution over bf16 rows.
#include "gdp_conv_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_conv_fwd<__nv_bfloat16>(ConvProblem &, int, int, bool, cudaStream_t);
template cudaError_t launch_conv_states<__nv_bfloat16>(const ConvProblem &, int, cudaStream_t);
template cudaError_t launch_conv_step<__nv_bfloat16>(const ConvProblem &, int, cudaStream_t);
template cudaError_t launch_conv_bwd<__nv_bfloat16>(ConvProblem &, int, int, cudaStream_t);
}  // namespace layer
}  // namespace gdp
