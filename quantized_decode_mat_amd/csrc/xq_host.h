// xq_host.h — what the files of the C ABI share: refusals and common gates
// (defined in xq_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/xq.h"

namespace xq {
namespace host {

// Sets the thread's error text and returns `s`; ok() clears it.
xq_status fail(xq_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
xq_status ok();
// The current device is gfx950.
xq_status check_device();
xq_status check_workspace(const void* ws, size_t ws_bytes, size_t need, const char* query);
xq_status check_workspace_align(const void* ws, size_t need);
xq_status launched(hipError_t e, const char* what);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace host
}  // namespace xq
