// Host helpers shared by the C-ABI entry points (wkv7_api.cpp, seq_api.cpp):
// the thread's error message, pointer checks, the architecture check and the
// report of a launch.  Defined in wkv7_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace wkv7 {

extern thread_local char g_last_error[512];

// Record the calling thread's message; returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A named device range [p, p + bytes) for the overlap checks.
struct Span {
    const void* p;
    int64_t bytes;
    const char* name;
};
bool overlap(const void* a, int64_t na, const void* b, int64_t nb);
int check_workspace_disjoint(const void* ws, int64_t need, const Span* spans, int n);

// The current device is a gfx950 (looked up once per device).
int check_device();
int finish_launch(hipError_t e, const char* what);

}  // namespace wkv7
