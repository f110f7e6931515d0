// The delta scan's gradients of all chunks at once, both storage types.
#include "ssm_delta_kernel.h"

namespace ssm {

hipError_t launch_delta_grad_bf16(const deltak::DeltaGradDev& d, bool vec, hipStream_t st) {
  return deltak::launch_grad_io<dev::BF16>(d, vec, st);
}
hipError_t launch_delta_grad_f32(const deltak::DeltaGradDev& d, bool vec, hipStream_t st) {
  return deltak::launch_grad_io<dev::F32>(d, vec, st);
}

}  // namespace ssm
