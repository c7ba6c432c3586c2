// runtime.hpp -- host helpers shared by the entry points (defined in dg.cpp).
#pragma once
#include <cstddef>
#include <cstdint>
#include <mutex>

#include <hip/hip_runtime_api.h>

#include "dg.h"
#include "plan.hpp"

namespace dg {

// An environment switch: set to a value that starts with 1.
bool env_on(const char *name);

// The current device's description, cached per device.  require: a missing
// device is an error rather than the default description.
dg_status current_device(Device *d, bool require);

// DG_ERR_POINTER unless p is device memory (null passes).
dg_status check_pointer(const void *p);

// The split-K blocks of one call (null when the plan needs none), locked while
// it lives: FP32 partial sums and arrival counters (zero on entry, to be left
// so) of the current device and the stream.
struct WsLease {
    std::unique_lock<std::mutex> lock;
    float *ws = nullptr;
    int *counters = nullptr;
};
hipError_t lease_workspace(hipStream_t stream, size_t bytes, size_t ncounters, WsLease *out);

}  // namespace dg
