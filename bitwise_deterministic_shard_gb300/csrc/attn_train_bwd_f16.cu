// The training attention's backward passes in f16.
#include "attn_train_bwd.cuh"

namespace detattn {
template cudaError_t ta_dkv<64, false>(const TaArgs&, cudaStream_t);
template cudaError_t ta_dkv<128, false>(const TaArgs&, cudaStream_t);
template cudaError_t ta_dq<64, false>(const TaArgs&, cudaStream_t);
template cudaError_t ta_dq<128, false>(const TaArgs&, cudaStream_t);
}  // namespace detattn
