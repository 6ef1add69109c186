// The causal convolution's kernels for bfloat16 activations.
#include "causal_conv_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_causal_conv<BF16>(const ConvArgs&, int, hipStream_t);
template hipError_t launch_causal_conv_grad<BF16>(const ConvArgs&, int, hipStream_t);
template hipError_t launch_causal_conv_step<BF16>(const ConvArgs&, int, hipStream_t);
}  // namespace seq
}  // namespace canon
