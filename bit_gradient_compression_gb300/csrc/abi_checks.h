// Host-side argument checks shared by the entry points (defined in abi.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "loco.h"

namespace loco {

// Records the text for loco_last_error() and returns st.
loco_status fail(loco_status st, const char* fmt, ...);

// Null and alignment check (no CUDA call).
loco_status check_ptr(const void* p, size_t align, const char* name);

// A list of buffers checked together: every null/alignment rule first, then
// the device-memory and extent rules, so the status does not depend on which
// buffer happens to be listed first.
struct BufCheck {
  const void* p;
  size_t bytes;
  size_t align;
  const char* name;
};
loco_status check_buffers(const BufCheck* b, int count);

// Whether two byte ranges share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb);

// LOCO_OK (and no error text), or LOCO_ERR_CUDA with the error's text.
loco_status launch_result(cudaError_t e, const char* what);

}  // namespace loco
