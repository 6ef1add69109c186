// The gated linear recurrence's kernels for bfloat16 activations.
#include "recurrence_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_recurrence<BF16>(const RecurArgs&, hipStream_t);
template hipError_t launch_recurrence_grad<BF16>(const RecurArgs&, hipStream_t);
template hipError_t launch_recurrence_step<BF16>(const RecurArgs&, hipStream_t);
}  // namespace seq
}  // namespace canon
