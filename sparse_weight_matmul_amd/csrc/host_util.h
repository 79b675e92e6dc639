// What the files of the C ABI share: error mapping, the dispatch log and the
// device's CU count.
#pragma once

#include <hip/hip_runtime.h>

#include "swm.h"

namespace swm {

// SWM_LOG=1: one stderr line per dispatch decision.
__attribute__((format(printf, 1, 2))) void swm_log(const char* fmt, ...);

// Remembers the error for swm_last_hip_error.
swm_status hip_fail(hipError_t e);

int num_cus(int dev);

}  // namespace swm

#define SWM_HIP(expr)                               \
  do {                                              \
    hipError_t e_ = (expr);                         \
    if (e_ != hipSuccess) return swm::hip_fail(e_); \
  } while (0)
