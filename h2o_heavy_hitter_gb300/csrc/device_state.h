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

}  // namespace h2o
