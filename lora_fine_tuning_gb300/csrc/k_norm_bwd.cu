// The backward of the norms around a block without the weights' gradients.
#include "norm_bwd.cuh"

namespace lora {

cudaError_t launch_norm_bwd(NormBwd& p, int sms, cudaStream_t stream) { return launch_norm_bwd_form<false, false>(p, sms, stream); }

}  // namespace lora
