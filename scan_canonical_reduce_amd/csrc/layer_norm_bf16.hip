// The layer norm's kernels for bfloat16 activations.
#include "layer_norm_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_layer_norm<BF16, F32>(const NormArgs&, hipStream_t);
template hipError_t launch_layer_norm_grad<BF16, F32>(const NormArgs&, hipStream_t);
template hipError_t launch_layer_norm<BF16, BF16>(const NormArgs&, hipStream_t);
template hipError_t launch_layer_norm_grad<BF16, BF16>(const NormArgs&, hipStream_t);
}  // namespace seq
}  // namespace canon
