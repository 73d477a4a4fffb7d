// Log probability kernels instantiated for f32 logits.

#include "logprob.cuh"

namespace normk {

template cudaError_t launch_logprob<F32>(LogprobArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_logprob_grad<F32>(LogprobGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
