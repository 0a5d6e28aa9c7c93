// Host helpers shared by the C entry points (defined in spense_abi.cu): status
// codes with a message for the calling thread, alignment, the current device.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "spense.h"

namespace spense {

spense_status fail(spense_status code, const char* fmt, ...);
spense_status ok();
spense_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct DeviceInfo {
  int major = 0;
  int sms = 0;
};

// Current device's capability and SM count (cached per device).
spense_status current_device(int* dev, DeviceInfo* info);

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace spense
