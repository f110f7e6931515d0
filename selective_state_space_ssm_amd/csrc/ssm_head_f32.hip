// The head scan's chunk kernels for float32 storage (one source file per type: they compile side by side).
#include "ssm_head_kernel.h"

namespace ssm {

hipError_t launch_head_f32(const headk::HeadDev& p, int mode, bool wide, bool vec, hipStream_t st) {
  return headk::launch_head_io<dev::F32>(p, mode, wide, vec, st);
}

}  // namespace ssm
