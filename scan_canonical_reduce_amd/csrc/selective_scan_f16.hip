// The selective scan's forward kernels for float16 activations.
#include "selective_scan_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_selective_scan<F16>(const ScanArgs&, int64_t, hipStream_t);
template hipError_t launch_selective_scan_step<F16>(const ScanArgs&, int64_t, hipStream_t);
}  // namespace seq
}  // namespace canon
