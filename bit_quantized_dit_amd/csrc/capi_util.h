// Host helpers shared by the C-ABI front ends.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/w4a4.h"

namespace w4a4 {

constexpr size_t kAlign = 256;   // arrays inside a blob or workspace

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }
inline int dev_status(hipError_t e) { return e == hipSuccess ? W4A4_OK : W4A4_ERR_DEVICE; }

}  // namespace w4a4
