// The gated linear recurrence's kernels for float16 activations.
#include "recurrence_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_recurrence<F16>(const RecurArgs&, hipStream_t);
template hipError_t launch_recurrence_grad<F16>(const RecurArgs&, hipStream_t);
template hipError_t launch_recurrence_step<F16>(const RecurArgs&, hipStream_t);
}  // namespace seq
}  // namespace canon
