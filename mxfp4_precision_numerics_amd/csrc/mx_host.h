// mx_host.h -- host-side helpers of the entry points (launch status, grids,
// alignment checks).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mx.h"

namespace mx {

inline bool aligned_to(const void* p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The status of the launches since the error state was last cleared.
inline mx_status launch_status() { return hipGetLastError() == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

inline size_t type_bytes(mx_dtype t) { return t == MX_BF16 ? 2 : 4; }

}  // namespace mx
