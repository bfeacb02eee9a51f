// Error reporting and pointer checks shared by the C ABI's translation units.
#pragma once

#include "../../include/qlinear.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlapi {

// Records the thread's error text and returns st.
ql_status fail(ql_status st, const char* fmt, ...);
ql_status hip_fail(hipError_t e, const char* what);

inline bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

}  // namespace qlapi
