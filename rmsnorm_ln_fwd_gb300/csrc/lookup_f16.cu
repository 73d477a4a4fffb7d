// Token lookup kernels instantiated for fp16 rows.

#include "lookup.cuh"

namespace normk {

template cudaError_t launch_lookup<F16>(LookupArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup_grad<F16>(LookupGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
