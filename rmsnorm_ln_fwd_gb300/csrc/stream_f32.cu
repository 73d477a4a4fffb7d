// Block join and token lookup kernels instantiated for fp32 rows.

#include "join_bwd.cuh"
#include "join_fwd.cuh"
#include "lookup.cuh"

namespace normk {

template cudaError_t launch_join<F32>(JoinArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_join_grad<F32>(JoinGradArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup<F32>(LookupArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup_grad<F32>(LookupGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
