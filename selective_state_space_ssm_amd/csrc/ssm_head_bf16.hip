// The head scan's chunk kernels for bfloat16 storage (one source file per type: they compile side by side).
#include "ssm_head_kernel.h"

namespace ssm {

hipError_t launch_head_bf16(const headk::HeadDev& p, int mode, bool wide, bool vec, hipStream_t st) {
  return headk::launch_head_io<dev::BF16>(p, mode, wide, vec, st);
}

}  // namespace ssm
