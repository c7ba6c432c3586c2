// runtime.hpp -- host helpers shared by the entry points (defined in dg.cpp).
#pragma once
#include <cstdint>

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

}  // namespace dg
