// The backward of the norms around a block from what was kept in 8 bits, without the weights' gradients.
#include "norm_bwd.cuh"

namespace lora {

cudaError_t launch_norm_bwd8(NormBwd& p, int sms, cudaStream_t stream) { return launch_norm_bwd_form<false, true>(p, sms, stream); }

}  // namespace lora
