// The layer norm's kernels for 32-bit activations.
#include "layer_norm_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_layer_norm<F32, F32>(const NormArgs&, hipStream_t);
template hipError_t launch_layer_norm_grad<F32, F32>(const NormArgs&, hipStream_t);
}  // namespace seq
}  // namespace canon
