// api_common.h -- what the C-ABI sources share: the device check and the
// argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bsr.h"

namespace bsr {

// BSR_OK if the calling thread's current device is a gfx950 GPU (cached per
// device), else BSR_EDEVICE.
int check_device();

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool k_ok(uint32_t k) { return k != 0 && k % 32 == 0; }

// Grids stay below 2^31 workgroups.
constexpr uint64_t kMaxGrid = (1ull << 31) - 1;

inline int launched(hipError_t e) { return e == hipSuccess ? BSR_OK : BSR_ELAUNCH; }

}  // namespace bsr
