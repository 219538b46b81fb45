// Helpers that the files of C entry points share.
#pragma once
#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

#include "w8a8.h"

namespace w8a8 {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t v) { return (v + 255u) & ~size_t(255u); }
inline w8a8_status launched(hipError_t e) { return e == hipSuccess ? W8A8_OK : W8A8_ERR_LAUNCH; }
// W8A8_OK when the current HIP device is a gfx950 (cached per device).
w8a8_status check_device();

}  // namespace w8a8
