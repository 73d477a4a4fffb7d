// Per-head norm and rotation kernels instantiated for bf16 rows.

#include "heads.cuh"

namespace normk {

template cudaError_t launch_head_rotary<BF16>(HeadArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_head_rotary_grad<BF16>(HeadArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
