// Token lookup kernels instantiated for fp32 rows.

#include "lookup.cuh"

namespace normk {

template cudaError_t launch_lookup<F32>(LookupArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup_grad<F32>(LookupGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
