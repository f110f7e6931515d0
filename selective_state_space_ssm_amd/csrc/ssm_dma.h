// Loads straight into LDS (16 bytes a lane) for kernels that count and wait for
// them themselves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_device.h"

namespace ssm {
namespace dev {

typedef __attribute__((address_space(3))) void lds_void;

// Buffer descriptor words for dma16: base, stride 0, size in bytes.
__device__ __forceinline__ u32x4 dma_desc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  u32x4 d;
  d.x = static_cast<uint32_t>(a);
  d.y = static_cast<uint32_t>(a >> 32) & 0xffffu;
  d.z = bytes;
  d.w = static_cast<uint32_t>(kRsrcWord3);
  return d;
}

// 16 bytes per lane from the buffer at byte offset voff (past the size:
// zeros) into LDS at lds + 16 * lane.  Written as inline asm so that the
// compiler does not count it: it would otherwise wait for every load in
// flight before the next LDS read, which undoes the pipeline.  The kernel
// waits for these loads itself (vmcnt before the barrier of the step that
// reads the stage, and all of them before the workgroup ends).  M0 holds
// the LDS address; one wait state separates its write from the load that
// reads it.  Nothing else in the kernel uses M0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const u32x4& d, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(d)
               : "memory", "m0");
}
#pragma clang diagnostic pop

}  // namespace dev
}  // namespace ssm
