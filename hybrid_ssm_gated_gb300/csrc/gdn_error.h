// gdn_error.h -- the error record behind gdn_last_error_string(), for the files with entry points.
#pragma once

#include <cuda_runtime.h>

namespace gdn {

// Record a message (printf form) and return `code`.
int fail(int code, const char* fmt, ...);
// A launch's result as a return code.
int launched(cudaError_t e, const char* what);
// The last failure's message on this thread.
const char* last_error();

}  // namespace gdn
