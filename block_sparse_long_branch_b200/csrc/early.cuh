// early.cuh -- kernels that start while the one before them in the stream ends.
#pragma once

#include <utility>

#include "kernels.h"
#include "sm100.cuh"

namespace msa {

// A launch that may start while the kernel before it in the stream still runs
// (the kernel calls pdl_wait before it touches what that one writes).
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kern)(Params...), int grid, int threads, int smem, cudaStream_t s,
                         Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Zeroes the first `words` words of a workspace: the error word, and what follows
// it.  A kernel of its own, not a memset, because the kernel behind it may start
// early: it finds all earlier work of the stream done, and waits for the zeros only
// before it records an error, takes a ticket or ends (decode of one request of 4K:
// 18.5 -> 16.4 us back to back).  It costs the host 2 us more than a memset does.
static __global__ void __launch_bounds__(256) clear_kernel(uint4* p, int64_t words) {
  pdl_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (4 * i < words) p[i] = make_uint4(0, 0, 0, 0);
}
// words: a multiple of 4
static inline cudaError_t launch_clear(void* p, int64_t words, cudaStream_t s) {
  clear_kernel<<<(unsigned)((words / 4 + 255) / 256), 256, 0, s>>>(static_cast<uint4*>(p), words);
  return cudaGetLastError();
}

// an error recorded by a kernel that launch_early put behind launch_clear
__device__ __forceinline__ void record_error_early(uint32_t* err, uint32_t code) {
  pdl_wait();
  record_error(err, code);
}

}  // namespace msa
