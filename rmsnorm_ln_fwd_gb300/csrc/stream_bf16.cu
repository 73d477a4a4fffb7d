// Block join and token lookup kernels instantiated for bf16 rows.

#include "join_bwd.cuh"
#include "join_fwd.cuh"
#include "lookup.cuh"

namespace normk {

template cudaError_t launch_join<BF16>(JoinArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_join_grad<BF16>(JoinGradArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup<BF16>(LookupArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_lookup_grad<BF16>(LookupGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
