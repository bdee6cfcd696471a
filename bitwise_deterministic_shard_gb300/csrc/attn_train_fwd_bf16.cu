// The training attention's forward pass in bf16.
#include "attn_train_fwd.cuh"

namespace detattn {
template cudaError_t ta_forward<64, true>(const TaArgs&, cudaStream_t);
template cudaError_t ta_forward<128, true>(const TaArgs&, cudaStream_t);
}  // namespace detattn
