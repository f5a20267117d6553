// check.h -- what the fusions' and the operators' entry points share: the
// error message of the calling thread and the check of a caller's buffer.
#pragma once

#include <hip/hip_runtime_api.h>

#include <string>

#include "hlofusion.h"

namespace hf {

void set_error(const std::string &m);  // what hf_last_error returns
hf_status hip_error(hipError_t e, const char *what);

// A buffer must be device memory of `device` (or managed memory), with its
// whole extent inside one allocation: anything else is rejected, before a
// kernel could fault on it.
bool check_buffer(const void *p, size_t bytes, int device, const char *owner, const std::string &what);

}  // namespace hf
