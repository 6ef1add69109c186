// The selective scan's forward kernels for float32 activations.
#include "selective_scan_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_selective_scan<F32>(const ScanArgs&, int64_t, hipStream_t);
template hipError_t launch_selective_scan_step<F32>(const ScanArgs&, int64_t, hipStream_t);
}  // namespace seq
}  // namespace canon
