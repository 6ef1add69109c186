// The causal convolution's kernels for float16 activations.
#include "causal_conv_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_causal_conv<F16>(const ConvArgs&, int, hipStream_t);
template hipError_t launch_causal_conv_grad<F16>(const ConvArgs&, int, hipStream_t);
template hipError_t launch_causal_conv_step<F16>(const ConvArgs&, int, hipStream_t);
}  // namespace seq
}  // namespace canon
