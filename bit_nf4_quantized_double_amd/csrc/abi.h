// Host-side helpers of the extern "C" entry points: the status and message of
// a failure, and alignment.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <string>

#include <hip/hip_runtime.h>

namespace qlora {

// Records the calling thread's message (qlora_last_error) and returns status.
int fail(int status, const std::string& msg);
int hip_fail(hipError_t e, const char* where);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace qlora
