// Block join and token lookup kernels instantiated for fp16 rows.

#include "join_bwd.cuh"
#include "join_fwd.cuh"
#include "lookup.cuh"

namespace normk {

template cudaError_t launch_join<F16>(JoinArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_join_grad<F16>(JoinGradArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup<F16>(LookupArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup_grad<F16>(LookupGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
