// Block join forward kernels instantiated for fp32 rows.

#include "join_fwd.cuh"

namespace normk {

template cudaError_t launch_join<F32>(JoinArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
