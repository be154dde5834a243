// fa_host.h -- host-side helpers of the C-ABI front end that every translation
// unit with entry points shares (defined in fa_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"

namespace fa_host {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, or nullptr when the driver has none
EncodeTiledFn encode_fn();

// The current device with its one-time set-up done: FA_OK with its index and
// multiprocessor count, else the status an entry point returns.
int current_device(int* dev, int* sms);

// device (or managed) memory that kernels on `dev` may use
bool is_device_pointer(const void* p, int dev);

// device address of the status word on `dev` (nullptr if it cannot be looked
// up); the first lookup on a device must not run inside a stream capture
unsigned int* status_word(int dev);

// Status of a launch by what the launch itself returned: an error that an earlier call of the process left behind
// is not this one's, and a call that reports a failure has turned nothing in place.
inline int launched(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  cudaGetLastError();
  return FA_ERR_LAUNCH;
}

constexpr int kMaxDevices = 64;

}  // namespace fa_host
