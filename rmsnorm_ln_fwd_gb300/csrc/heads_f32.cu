// Per-head norm and rotation kernels instantiated for f32 rows.

#include "heads.cuh"

namespace normk {

template cudaError_t launch_head_rotary<F32>(HeadArgs, const DeviceInfo&, cudaStream_t);
template cudaError_t launch_head_rotary_grad<F32>(HeadArgs, const DeviceInfo&, cudaStream_t);

}  // namespace normk
