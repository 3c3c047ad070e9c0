// api_common.hpp -- error reporting and pointer checks shared by the files of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

// Record the thread's error text and return s; clear it and return QMM_OK.
qmm_status fail(qmm_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
qmm_status ok();
qmm_status hip_fail(hipError_t e, const char* what);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace qmm
