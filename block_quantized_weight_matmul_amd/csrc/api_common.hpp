// api_common.hpp -- error reporting and argument checks shared by the files of the C ABI.
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

typedef long long ll;

inline hipStream_t stream_of(qmm_stream_t s) { return reinterpret_cast<hipStream_t>(s); }
inline bool dtype_ok(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
inline int64_t size_of(int t) { return t == QMM_F32 ? 4 : 2; }

inline qmm_status check_dtype(int t, const char* what) {
  return dtype_ok(t) ? QMM_OK : fail(QMM_E_TYPE, "unknown %s dtype %d", what, t);
}
inline qmm_status check_ptr(const void* p, uintptr_t align, const char* what) {
  if (!p) return fail(QMM_E_ARG, "%s is NULL", what);
  if (!aligned(p, align)) return fail(QMM_E_ALIGN, "%s must be %d-byte aligned", what, static_cast<int>(align));
  return QMM_OK;
}
inline qmm_status check_range(int64_t v, int64_t lo, int64_t hi, const char* what) {
  return v >= lo && v <= hi ? QMM_OK
                            : fail(QMM_E_SHAPE, "%s=%lld outside [%lld, %lld]", what, static_cast<ll>(v),
                                   static_cast<ll>(lo), static_cast<ll>(hi));
}
inline qmm_status check_ws(const void* ws, size_t have, size_t need, const char* what) {
  if (need == 0) return QMM_OK;
  if (!ws) return fail(QMM_E_ARG, "%s is NULL; this call needs %zu bytes", what, need);
  if (have < need) return fail(QMM_E_ARG, "%s holds %zu bytes; this call needs %zu", what, have, need);
  if (!aligned(ws, 16)) return fail(QMM_E_ALIGN, "%s must be 16-byte aligned", what);
  return QMM_OK;
}

#define QMM_TRY(expr)                     \
  do {                                    \
    const qmm_status s_ = (expr);         \
    if (s_ != QMM_OK) return s_;          \
  } while (0)

}  // namespace qmm
