// internal.h -- what the library's entry points share: the thread's error text
// and stream, and the library workspace (gemm_api.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <mutex>
#include <string>

namespace dgw {

// Set the thread's error text and return `code`.
int set_error(int code, const std::string &msg);
int set_hip_error(hipError_t e, const char *what);
void clear_error();

// The stream that a call's `stream` argument names: the calling thread's
// (gemm_set_stream) for NULL, HIP's null stream for GEMM_NULL_STREAM.
hipStream_t call_stream(void *stream);

// Compute units of the current device.
int current_device_cus(int *out);

// At least `bytes` of the current device's library workspace.  Refused while
// `stream` is being captured if the workspace would have to grow.  `lock` receives
// the library's lock, which the caller keeps until its last kernel is enqueued:
// until then no other thread's call uses the workspace, and gemm_release() waits.
int library_workspace(int64_t bytes, hipStream_t stream, void **out, std::unique_lock<std::mutex> *lock);

}  // namespace dgw
