// Block join gradient kernels instantiated for fp16 rows.

#include "join_bwd.cuh"

namespace normk {

template cudaError_t launch_join_grad<F16>(JoinGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
