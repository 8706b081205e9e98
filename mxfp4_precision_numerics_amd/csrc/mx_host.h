// mx_host.h -- host-side helpers of the entry points (launch status, grids,
// alignment checks).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mx.h"

namespace mx {

inline bool aligned_to(const void* p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// (The runtime's host min and max are of 32 bits, whatever they are given.)
__host__ __device__ __forceinline__ int64_t lesser(int64_t a, int64_t b) { return b < a ? b : a; }
__host__ __device__ __forceinline__ int64_t greater(int64_t a, int64_t b) { return a < b ? b : a; }

// The status of the launches since the error state was last cleared.
inline mx_status launch_status() { return hipGetLastError() == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

inline size_t type_bytes(mx_dtype t) { return t == MX_BF16 ? 2 : 4; }

}  // namespace mx
