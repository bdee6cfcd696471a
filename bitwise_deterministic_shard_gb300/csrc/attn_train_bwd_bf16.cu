// The training attention's backward passes in bf16.
#include "attn_train_bwd.cuh"

namespace detattn {
template cudaError_t ta_dkv<64, true>(const TaArgs&, cudaStream_t);
template cudaError_t ta_dkv<128, true>(const TaArgs&, cudaStream_t);
template cudaError_t ta_dq<64, true>(const TaArgs&, cudaStream_t);
template cudaError_t ta_dq<128, true>(const TaArgs&, cudaStream_t);
}  // namespace detattn
