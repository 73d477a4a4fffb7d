// Per-head norm and rotation kernels instantiated for f16 rows.

#include "heads.cuh"

namespace normk {

template cudaError_t launch_head_rotary<F16>(HeadArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_head_rotary_grad<F16>(HeadArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
