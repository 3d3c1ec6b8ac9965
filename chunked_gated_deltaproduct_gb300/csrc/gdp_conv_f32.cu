// gdp_conv_f32.cu -- the short causal convolution over f32 rows.
#include "gdp_conv_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_conv_fwd<float>(ConvProblem &, int, int, bool, cudaStream_t);
template cudaError_t launch_conv_states<float>(const ConvProblem &, int, cudaStream_t);
template cudaError_t launch_conv_step<float>(const ConvProblem &, int, cudaStream_t);
template cudaError_t launch_conv_bwd<float>(ConvProblem &, int, int, cudaStream_t);
}  // namespace layer
}  // namespace gdp
