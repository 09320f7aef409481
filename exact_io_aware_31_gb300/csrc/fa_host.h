// Host-side helpers shared by the files that define C ABI entry points.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

namespace fa {

// Facts about the current device plus the status word's address in the
// current context.
struct DeviceInfo {
  int sms = 0;
  bool sm103 = false;
  int* status = nullptr;  // device address of g_device_status in the current context
};

// FA_OK and *out filled, FA_ERR_UNSUPPORTED off sm_103, or FA_ERR_CUDA.
int device_info(DeviceInfo* out);

// cuTensorMapEncodeTiled; valid once device_info() has succeeded.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// scale * log2(e), its magnitude floored at 1e-30 so that a masked score
// (-inf) times |c2| stays -inf when scale == 0.  For finite scores |s| < 1e8
// the floor changes 2^(s * c2) by less than one fp32 ulp of 1, so scale == 0
// still gives exact uniform attention.  The sign is kept: the tensor-core
// kernels compute S negated for a negative scale and use |c2| after it.
inline float log2_scale(float scale) {
  const float c2 = scale * 1.4426950408889634f;
  return std::fabs(c2) > 1e-30f ? c2 : std::copysign(1e-30f, c2);
}

}  // namespace fa
