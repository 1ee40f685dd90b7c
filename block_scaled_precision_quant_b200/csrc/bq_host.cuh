// bq_host.cuh -- host state that the translation units of libbq share: the
// per-device facts and error word, and the tensor-map encoder (both defined
// in bq_api.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdint.h>

namespace bqh {

constexpr int kMaxDevices = 64;

struct Device {
  int index = 0;
  int num_sms = 0;
  int* err = nullptr;  // the library's device error word on this device
};

// The current device: BQ_OK, BQ_ERR_ARCH (not compute capability 10.0) or
// BQ_ERR_CUDA.
__attribute__((visibility("hidden"))) int current_device(Device* d);

// cuTensorMapEncodeTiled, or nullptr if the driver has no such entry.
__attribute__((visibility("hidden"))) PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace bqh
