// What the files that hold C entry points share (defined in sgemm_f32.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace sgemm {

// Records e for sgemm_f32_last_hip_error; returns SGEMM_ERR_HIP.
int hip_fail(hipError_t e);
// SGEMM_OK if `bytes` bytes from p on lie in one allocation of device dev,
// else SGEMM_ERR_POINTER; lo and hi, if given, receive where that allocation
// begins and ends.  bytes <= 0: nothing to check.
int check_device_range(const void *p, int64_t bytes, int dev, uintptr_t *lo = nullptr, uintptr_t *hi = nullptr);

}  // namespace sgemm
