// Token lookup kernels instantiated for bf16 rows.

#include "lookup.cuh"

namespace normk {

template cudaError_t launch_lookup<BF16>(LookupArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup_grad<BF16>(LookupGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
