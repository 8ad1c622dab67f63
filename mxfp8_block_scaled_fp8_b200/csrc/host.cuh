// host.cuh -- host-side helpers shared by the library's translation units:
// device facts, error bookkeeping and launches.
#pragma once

#include "fp8mm.h"

#include <cuda_runtime.h>

#include <cstdint>

namespace fp8mm {

struct DeviceInfo {
  int device = -1;
  int sms = 0;
  bool sm100 = false;
};

// Keeps the CUDA error for fp8mm_last_cuda_error and gives FP8MM_ERR_LAUNCH.
fp8mm_status cuda_fail(cudaError_t e);
// Facts of the current device (cached); FP8MM_ERR_UNSUPPORTED unless sm_100.
fp8mm_status current_device(DeviceInfo* info);
// Opt a kernel into its dynamic shared memory size, once per device.
fp8mm_status ensure_smem(const void* kernel, int bytes, int dev);
// Limit of the bounded waits inside kernels.
uint64_t wait_timeout_ns();
// Returns and clears the device error word of the cache operators' kernels
// (each translation unit has its own word); the device must be idle.
unsigned int kv_take_device_error();

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Launch with programmatic stream serialisation (the kernel may begin while
// the preceding kernel on the stream finishes; it waits for it in-kernel).
template <typename... KArgs, typename... Args>
fp8mm_status launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                        Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e == cudaSuccess ? FP8MM_OK : cuda_fail(e);
}

inline fp8mm_status launched() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FP8MM_OK : cuda_fail(e);
}

}  // namespace fp8mm
