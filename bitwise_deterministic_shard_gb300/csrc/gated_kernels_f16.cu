// The gated feed-forward kernels, f16 operands.
#include "gated_kernels.cuh"

namespace detattn {
template cudaError_t gl_forward<false>(const GlArgs&, cudaStream_t);
template cudaError_t gl_backward<false>(const GlArgs&, cudaStream_t);
template cudaError_t gl_few<false>(const GlFewArgs&, cudaStream_t);
template cudaError_t gl_scale<false>(const GlScaleArgs&, cudaStream_t);
}  // namespace detattn
