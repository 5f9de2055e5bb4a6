// Errors at the C boundary: an entry point's body runs inside guarded(), which
// turns failures into a status and the thread's message (lopt_last_error).
#pragma once

#include <hip/hip_runtime.h>

#include <exception>
#include <new>
#include <string>

#include "../../include/lopt.h"

namespace lopt {

// The calling thread's message, defined in lopt_api.cpp.
std::string& last_error();

struct ApiError {
  lopt_status code;
  std::string msg;
};

[[noreturn]] inline void fail(lopt_status code, const std::string& msg) { throw ApiError{code, msg}; }

inline void hip_check(hipError_t e, const char* what) {
  if (e != hipSuccess) fail(LOPT_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

template <class F>
lopt_status guarded(F&& f) {
  try {
    f();
    last_error().clear();
    return LOPT_OK;
  } catch (const ApiError& e) {
    last_error() = e.msg;
    return e.code;
  } catch (const std::bad_alloc&) {
    last_error() = "host allocation failed";
    return LOPT_ERR_HIP;
  } catch (const std::exception& e) {
    last_error() = e.what();
    return LOPT_ERR_HIP;
  } catch (...) {
    last_error() = "unknown error";
    return LOPT_ERR_HIP;
  }
}

}  // namespace lopt
