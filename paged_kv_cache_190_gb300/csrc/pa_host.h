// Host state shared by the C ABI's translation units (defined in capi.cu).
#pragma once

#include <cstdint>

namespace pa {

// SM count of the current device, <= 0 when there is none.
int current_sm_count();
// Bound on each pipeline wait in polls, < 0: the kernels' default.
int64_t wait_limit();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

}  // namespace pa
