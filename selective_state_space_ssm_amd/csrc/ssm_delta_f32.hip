// The delta scan's walks over the length for float32 storage.
#include "ssm_delta_kernel.h"

namespace ssm {

hipError_t launch_delta_f32(const deltak::DeltaDev& p, const deltak::DeltaDev& r, int pass, bool vec, hipStream_t st) {
  return deltak::launch_pass_io<dev::F32>(p, r, pass, false, vec, st);
}

}  // namespace ssm
