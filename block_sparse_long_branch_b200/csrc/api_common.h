// api_common.h -- helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/msa.h"

namespace msa {

constexpr size_t kHeader = 256;  // device error word + reserved

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// A failed launch is reported through the status; the runtime's last-error
// slot is cleared so that the caller's next, unrelated CUDA call does not
// see it again (a sticky error stays sticky regardless).
inline msa_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MSA_OK;
  (void)cudaGetLastError();
  return MSA_ERR_CUDA;
}

// launches of this host thread's last call (msa_last_launch_count)
void set_launch_count(int n);

// workspace of the full-attention operators (api_dense.cu)
msa_status_t dense_workspace_size(const msa_config_t* cfg, msa_op_t op, int64_t n_tokens,
                                  int32_t batch, size_t* bytes);

}  // namespace msa
