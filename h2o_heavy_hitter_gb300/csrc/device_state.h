// Per-device host state of the tensor-core kernels: the tensor-map encoder, the
// SM count and the shared-memory opt-ins.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>

namespace h2o {

// cuTensorMapEncodeTiled, or null where the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// SM count of the current device (one persistent CTA per SM).
int num_sms();

constexpr int kMaxDevices = 64;

// Lets `kernel` use `bytes` of dynamic shared memory on the current device.
// The attribute is per device, so it is set once per device and epoch
// (forget_device_state starts a new one); opted_in[dev], one array per kernel,
// records the epoch in which it was set. Safe to call from several threads.
cudaError_t raise_smem_limit(const void* kernel, size_t bytes, int (&opted_in)[kMaxDevices]);

// A launch that may begin while the kernel before it drains: the kernel waits
// (grid_dependency_wait) before it touches what that one writes.
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, size_t smem,
                         cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(static_cast<unsigned>(threads));
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

}  // namespace h2o
