// Error reporting and pointer checks shared by the C entry points (defined in api.cu).
#pragma once

#include <cuda_runtime.h>

#include "gdnq.h"

namespace gdnq {

// Empties the calling thread's last-error message; every entry point begins with it.
void clear_error();
// Stores the message and returns st.
gdn_status fail(gdn_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gdn_status cuda_fail(cudaError_t e, const char* where);
// p is not null and aligned to `align` bytes (a power of two).
gdn_status need_ptr(const void* p, const char* name, unsigned align = 16);

}  // namespace gdnq
