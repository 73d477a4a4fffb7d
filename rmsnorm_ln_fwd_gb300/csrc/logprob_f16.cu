// Log probability kernels instantiated for f16 logits.

#include "logprob.cuh"

namespace normk {

template cudaError_t launch_logprob<F16>(LogprobArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_logprob_grad<F16>(LogprobGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
