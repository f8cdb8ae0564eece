// Host helpers that the C entry points share: the calling thread's error text
// (defined in pkv_api.cu), the SM count, and alignment checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

// Records the message for pkv_last_error() and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message and returns PKV_OK.
int ok();
int cuda_fail(cudaError_t e, const char* what);
// SM count of the current device (cached per device).
int num_sms();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t div_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace pkv
