// dependent.cuh -- what the short calls around verification share: programmatic dependent launches,
// the status word's reset beside them, and bulk copies out of shared memory.
#pragma once

#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

// Lets the next kernel start beside this one, then waits until the work before this one is done and
// visible; everything a kernel shares with other work comes after it.  The loads that follow are
// ordinary ones: the read-only path wants memory that nobody writes while the kernel is resident.
__device__ __forceinline__ void dependent_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches `kernel` as a programmatic dependent: it may start while the kernel before it on the
// stream ends, and waits for that (dependent_start) before it touches what others wrote or read.
template <typename... KArgs, typename... Args>
inline sv_status launch_dependent(void (*kernel)(KArgs...), unsigned grid, unsigned threads,
                                  size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Sets the status word (if any) to SV_OK ahead of kernels launched by launch_dependent: a kernel
// that starts and ends beside them, where a memset would sit between two of them (quantising 384
// rows of 2560 6.1 -> 4.8 us a call).
sv_status reset_status(int32_t* status, cudaStream_t s);

// Bulk copy shared -> global in the thread's bulk group (src, dst 16-byte aligned, bytes % 16 == 0),
// the group's commit, and the wait until all committed copies have read their source.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_addr(src)), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void bulk_group_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void bulk_group_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

}  // namespace sv
