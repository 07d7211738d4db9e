// Checks shared by the C ABI layers (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8bs.h"

namespace fp8bs {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The current device must be a gfx950 (MI355X / MI350X).  The answer is
// cached per device ordinal; hipGetDevice itself fails when no GPU exists.
fp8bs_status check_device();

inline fp8bs_status launched(hipError_t e) { return e == hipSuccess ? FP8BS_OK : FP8BS_ERR_LAUNCH; }

}  // namespace fp8bs
