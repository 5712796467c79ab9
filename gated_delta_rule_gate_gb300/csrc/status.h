// status.h -- status codes, the thread-local message and argument checks shared
// by the C entry points of libgdn (defined in gdn_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

// Records the message of the first failed check and returns `st`.
gdn_status fail(gdn_status st, const char *fmt, ...);
// Clears the message and returns GDN_OK.
gdn_status ok();
// GDN_OK, or GDN_ERR_CUDA with the runtime's message.
gdn_status cuda_status(cudaError_t e);

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace gdn
