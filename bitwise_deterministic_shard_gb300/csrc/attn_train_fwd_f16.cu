// The training attention's forward pass in f16.
#include "attn_train_fwd.cuh"

namespace detattn {
template cudaError_t ta_forward<64, false>(const TaArgs&, cudaStream_t);
template cudaError_t ta_forward<128, false>(const TaArgs&, cudaStream_t);
}  // namespace detattn
