// The selective scan's backward kernels for float16 activations.
#include "selective_scan_grad_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_selective_scan_grad<F16>(const ScanArgs&, int64_t, hipStream_t);
}  // namespace seq
}  // namespace canon
