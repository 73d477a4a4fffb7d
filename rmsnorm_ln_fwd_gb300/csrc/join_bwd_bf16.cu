// Block join gradient kernels instantiated for bf16 rows.

#include "join_bwd.cuh"

namespace normk {

template cudaError_t launch_join_grad<BF16>(JoinGradArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
