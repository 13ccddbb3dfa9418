// Error reporting shared by the files that implement the C ABI.
#pragma once

#include <cuda_runtime_api.h>
#include <stdint.h>

#include "fbob.h"
#include "internal.h"

namespace fbob {

// Record the text that fbob_last_error returns on this host thread; return s.
fbob_status fail(fbob_status s, const char* fmt, ...);
fbob_status cuda_fail(cudaError_t e, const char* where);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Status word, wait limit and test hooks for a launch on the current device.
fbob_status make_ctx(DevCtx* c);

}  // namespace fbob
