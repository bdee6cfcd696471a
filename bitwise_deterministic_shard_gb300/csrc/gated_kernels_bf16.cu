// The gated feed-forward kernels, bf16 operands.
#include "gated_kernels.cuh"

namespace detattn {
template cudaError_t gl_forward<true>(const GlArgs&, cudaStream_t);
template cudaError_t gl_backward<true>(const GlArgs&, cudaStream_t);
template cudaError_t gl_few<true>(const GlFewArgs&, cudaStream_t);
template cudaError_t gl_scale<true>(const GlScaleArgs&, cudaStream_t);
}  // namespace detattn
