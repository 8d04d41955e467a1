// api_internal.h -- declarations shared between the library's C-ABI translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd.h"

namespace ssd {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Every non-empty array must be non-NULL and aligned.
inline bool check_ptr(const void *p, int64_t elems, size_t align) {
  if (elems == 0) return true;
  return p != nullptr && aligned(p, align);
}

// The status of a call's last runtime call.  The runtime also keeps an error for whoever asks it next
// (cudaGetLastError), which would be the thread's next call here: it is cleared, so that each call answers for itself.
inline ssd_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}

ssd_status prefill_into_workspace(const ssd_dims *dims, ssd_dtype dtype, const void *x, const float *dt,
                                  const float *A, const void *B, const void *C, const float *D, int chunk,
                                  float *y, float *final_state, void *workspace, size_t workspace_bytes,
                                  ssd_stream_t stream);

}  // namespace ssd
