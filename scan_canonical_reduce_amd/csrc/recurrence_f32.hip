// The gated linear recurrence's kernels for 32-bit activations.
#include "recurrence_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_recurrence<F32>(const RecurArgs&, hipStream_t);
template hipError_t launch_recurrence_grad<F32>(const RecurArgs&, hipStream_t);
template hipError_t launch_recurrence_step<F32>(const RecurArgs&, hipStream_t);
}  // namespace seq
}  // namespace canon
