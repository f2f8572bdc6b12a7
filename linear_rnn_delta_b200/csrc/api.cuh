// Host helpers shared by the C ABI's translation units (kda_api.cu, linattn_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {
namespace api {

// Records the calling thread's error detail (kda_last_error_detail) and returns `code`.
int fail(int code, const char *fmt, ...);
int cuda_fail(cudaError_t e, const char *where);
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool head_dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

}  // namespace api
}  // namespace kda
