// Argument checks, error text and device check shared by the C ABI layers
// (mx_abi.cpp, mx_lm_abi.cpp); defined in mx_abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxfp8.h"

namespace mxabi {

// Records the message that mx_last_error() returns on this thread and
// returns st.
mx_status fail(mx_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mx_status check_device();
mx_status launched(hipError_t e, const char* what);

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace mxabi

#define MX_REQUIRE(cond, st, ...) \
  do {                            \
    if (!(cond)) return mxabi::fail(st, __VA_ARGS__); \
  } while (0)

#define MX_DEVICE()                          \
  do {                                       \
    mx_status st_ = mxabi::check_device();   \
    if (st_ != MX_OK) return st_;            \
  } while (0)

#define MX_CHECK(expr)              \
  do {                              \
    mx_status st_ = (expr);         \
    if (st_ != MX_OK) return st_;   \
  } while (0)
