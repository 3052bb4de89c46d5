// operators.h -- what the entry points of the operators share: checks of a
// descriptor's fields, the stream and its workspace, the result of a launch.
#pragma once

#include <new>
#include <string>

#include "context.h"

namespace gt {

// One failed check: the message for gt_last_error and the status to return.
inline gt_status refuse(gt_status st, const std::string& msg) {
  set_error(msg);
  return st;
}
inline gt_status invalid(const std::string& msg) { return refuse(GT_ERR_INVALID_ARG, msg); }

// A type of the 16- or 32-bit floating ones; `dflt` replaces a negative code.
inline gt_status float_type(int code, int dflt, const char* what, int* out) {
  const int t = code < 0 ? dflt : code;
  if (t < 0 || t > DT_E4M3) return invalid(std::string("unknown type of ") + what);
  if (t == DT_E4M3) return refuse(GT_ERR_UNSUPPORTED, std::string("e4m3 is not provided for ") + what);
  *out = t;
  return GT_OK;
}

inline gt_status leading(int64_t ld, int64_t row, const char* what, int64_t* out) {
  *out = ld > 0 ? ld : row;
  if (*out < row) return invalid(std::string(what) + ": leading dimension smaller than the row");
  return GT_OK;
}

// A matrix of `rows` rows must be addressable in 64-bit byte offsets, and
// its base aligned to its element.
inline gt_status spans(int64_t rows, int64_t ld, const char* what) {
  if (rows > 0 && ld > INT64_MAX / 8 / rows) return invalid(std::string(what) + " spans more than 64-bit offsets");
  return GT_OK;
}
inline gt_status operand(const void* p, bool required, int64_t rows, int64_t ld, int bytes, const char* what) {
  if (!p) return required ? invalid(std::string(what) + " is NULL") : GT_OK;
  if ((uintptr_t)p % bytes) return invalid(std::string(what) + " is not aligned to its element");
  return spans(rows, ld, what);
}

#define GT_CHECK(expr)                 \
  do {                                 \
    const gt_status _s = (expr);       \
    if (_s != GT_OK) return _s;        \
  } while (0)

inline hipStream_t stream_of(void* s) { return (hipStream_t)(s ? s : ctx().default_stream.load()); }

inline gt_status launched(int rc, const char* what) {
  if (rc == LS_OK) return GT_OK;
  if (rc == LS_UNSUPPORTED) return refuse(GT_ERR_UNSUPPORTED, std::string(what) + ": problem too large for the grid");
  return refuse(GT_ERR_HIP, std::string(what) + ": kernel launch failed");
}

// The stream's workspace for an operator.  Growing it allocates and clears
// memory, which a captured graph must not hold, so that is refused.
inline gt_status operator_workspace(DeviceState& d, hipStream_t stream, size_t bytes, void** ws, std::mutex** mu) {
  size_t have = 0;
  if (!d.fake) {
    if (find_workspace(d, (void*)stream, bytes, ws, &have, mu)) return GT_OK;
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    const bool asked = hipStreamIsCapturing(stream, &cs) == hipSuccess;
    if (!asked) hipGetLastError();  // the status says it; no later check should find it
    if ((!asked || cs != hipStreamCaptureStatusNone) && !workspace_ready(d, (void*)stream, bytes))
      return invalid("the workspace would have to grow under stream capture: make this call once before capturing");
  }
  return get_workspace(d, (void*)stream, bytes, ws, &have, mu);
}

// Nothing throws across the C boundary: an allocation that fails while a
// message or a workspace entry is made becomes a status.
template <class F, class D>
gt_status guarded(F f, const D* d) {
  try {
    return f(d);
  } catch (const std::bad_alloc&) {
    return GT_ERR_OOM;
  } catch (...) {
    return GT_ERR_HIP;
  }
}

}  // namespace gt
