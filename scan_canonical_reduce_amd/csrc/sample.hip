// The sampling's kernels.
#include "sample_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_sample<F32>(const SampleArgs&, hipStream_t);
template hipError_t launch_sample<BF16>(const SampleArgs&, hipStream_t);
template hipError_t launch_sample<F16>(const SampleArgs&, hipStream_t);
}  // namespace seq
}  // namespace canon
