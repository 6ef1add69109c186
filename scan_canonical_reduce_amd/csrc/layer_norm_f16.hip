// The layer norm's kernels for float16 activations.
#include "layer_norm_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_layer_norm<F16, F32>(const NormArgs&, hipStream_t);
template hipError_t launch_layer_norm_grad<F16, F32>(const NormArgs&, hipStream_t);
template hipError_t launch_layer_norm<F16, F16>(const NormArgs&, hipStream_t);
template hipError_t launch_layer_norm_grad<F16, F16>(const NormArgs&, hipStream_t);
}  // namespace seq
}  // namespace canon
