// host.hpp -- what the C entry points share on the host: argument checks,
// device facts, the per-(device, stream) scratch and the last HIP error.
// Defined in libred.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "libred.h"

namespace libred {

// Record `e` as the calling thread's last HIP error and return `code`.
red_status host_fail(hipError_t e, red_status code);
// Number of compute units of the current device.
red_status host_compute_units(int* dev, int* cu_count);
// The scratch buffer of (dev, stream), at least `bytes` long.
red_status host_scratch(int dev, hipStream_t stream, size_t bytes, void** out);

inline bool is_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace libred
