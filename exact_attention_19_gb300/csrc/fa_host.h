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

// 4-D map over a cache: (d, token of the page, K/V head, page), 128-byte
// swizzle, `rows` tokens x 64 elements per box.
inline bool make_cache_map(CUtensorMap* map, const void* ptr, int d, int page, int Hk, int n_pages, const long long* s,
                    int rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(Hk),
                        static_cast<cuuint64_t>(n_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(s[2]) * 2u, static_cast<cuuint64_t>(s[1]) * 2u,
                           static_cast<cuuint64_t>(s[0]) * 2u};
  cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(rows), 1u, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Status of a launch by what the launch itself returned: an error that an earlier call of the process left behind
// is not this one's, and a call that reports a failure has turned nothing in place.
inline int launched(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  cudaGetLastError();
  return FA_ERR_LAUNCH;
}

// Programmatic dependent launch: the kernel may be scheduled while the one ahead
// of it on the stream still runs, and waits on the device (griddepcontrol.wait)
// for what it needs of it.
template <typename K, typename... A>
int launch_kernel(K kernel, long long grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, kernel, args...));
}

constexpr int kMaxDevices = 64;

}  // namespace fa_host
