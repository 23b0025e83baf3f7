// Argument checks and error reporting shared by the extern "C" entry points
// (awq_api.hip, awq_api_serve.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "awq.h"

namespace awq {

// Records the calling thread's message for awq_last_error() and returns `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline int device_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return AWQ_OK;
  return fail(AWQ_ERROR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every device pointer an entry point takes must be 16-byte aligned (the
// kernels move 16-byte pieces, several of them straight into LDS); the first
// misaligned one is named in the error.  NULL entries (optional arguments
// left out) are skipped.
struct DevPtr {
  const void* p;
  const char* name;
};
inline int check_aligned(std::initializer_list<DevPtr> ptrs) {
  for (const DevPtr& d : ptrs)
    if (d.p != nullptr && !aligned16(d.p)) return fail(AWQ_ERROR_MISALIGNED, "%s must be 16-byte aligned", d.name);
  return AWQ_OK;
}

#define AWQ_REQUIRE(cond, status, ...) \
  do {                                 \
    if (!(cond)) return awq::fail(status, __VA_ARGS__); \
  } while (0)

#define AWQ_GUARD_BEGIN try {
#define AWQ_GUARD_END                                            \
  }                                                              \
  catch (...) {                                                  \
    return awq::fail(AWQ_ERROR_DEVICE, "unexpected C++ exception"); \
  }

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

inline int check_bits(int32_t bits) {
  AWQ_REQUIRE(bits == 4 || bits == 3, AWQ_ERROR_INVALID_VALUE, "bits must be 4 or 3 (got %d)", bits);
  return AWQ_OK;
}

inline int check_layer(int64_t N, int64_t K, int32_t group) {
  AWQ_REQUIRE(N >= 1 && K >= 1, AWQ_ERROR_INVALID_VALUE, "N and K must be >= 1 (got N=%lld K=%lld)", (long long)N,
              (long long)K);
  AWQ_REQUIRE(group == AWQ_GROUP, AWQ_ERROR_INVALID_VALUE, "group must be %d (got %d)", AWQ_GROUP, group);
  AWQ_REQUIRE(K % group == 0, AWQ_ERROR_INVALID_VALUE, "K=%lld is not a multiple of group %d", (long long)K, group);
  AWQ_REQUIRE(N < (int64_t(1) << 31) && K <= (int64_t(1) << 20), AWQ_ERROR_INVALID_VALUE,
              "N=%lld or K=%lld exceeds the supported range", (long long)N, (long long)K);
  return AWQ_OK;
}

}  // namespace awq
