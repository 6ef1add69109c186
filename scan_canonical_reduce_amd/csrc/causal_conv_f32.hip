// The causal convolution's kernels for float32 activations.
#include "causal_conv_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_causal_conv<F32>(const ConvArgs&, int, hipStream_t);
template hipError_t launch_causal_conv_grad<F32>(const ConvArgs&, int, hipStream_t);
template hipError_t launch_causal_conv_step<F32>(const ConvArgs&, int, hipStream_t);
}  // namespace seq
}  // namespace canon
