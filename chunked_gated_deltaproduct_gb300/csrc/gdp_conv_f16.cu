// gdp_conv_f16.cu -- the short causal convolution over f16 rows.
#include "gdp_conv_body.cuh"

namespace gdp {
namespace layer {
template cudaError_t launch_conv_fwd<__half>(ConvProblem &, int, int, bool, cudaStream_t);
template cudaError_t launch_conv_states<__half>(const ConvProblem &, int, cudaStream_t);
template cudaError_t launch_conv_step<__half>(const ConvProblem &, int, cudaStream_t);
template cudaError_t launch_conv_bwd<__half>(ConvProblem &, int, int, cudaStream_t);
}  // namespace layer
}  // namespace gdp
