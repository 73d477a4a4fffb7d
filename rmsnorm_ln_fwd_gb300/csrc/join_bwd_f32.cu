// Block join gradient kernels instantiated for fp32 rows.

#include "join_bwd.cuh"

namespace normk {

template cudaError_t launch_join_grad<F32>(JoinGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
