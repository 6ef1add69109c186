// The embedding lookup and gradient kernels.
#include "embedding_impl.hpp"

namespace canon {
namespace seq {
template hipError_t launch_embedding<F32>(const EmbedArgs&, hipStream_t);
template hipError_t launch_embedding<BF16>(const EmbedArgs&, hipStream_t);
template hipError_t launch_embedding<F16>(const EmbedArgs&, hipStream_t);
template hipError_t launch_embedding_grad<F32, F32>(const EmbedGradArgs&, hipStream_t);
template hipError_t launch_embedding_grad<BF16, F32>(const EmbedGradArgs&, hipStream_t);
template hipError_t launch_embedding_grad<BF16, BF16>(const EmbedGradArgs&, hipStream_t);
template hipError_t launch_embedding_grad<F16, F32>(const EmbedGradArgs&, hipStream_t);
template hipError_t launch_embedding_grad<F16, F16>(const EmbedGradArgs&, hipStream_t);
}  // namespace seq
}  // namespace canon
