// Log probability kernels instantiated for bf16 logits.

#include "logprob.cuh"

namespace normk {

template cudaError_t launch_logprob<BF16>(LogprobArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_logprob_grad<BF16>(LogprobGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
