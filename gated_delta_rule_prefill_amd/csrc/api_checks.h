// api_checks.h -- argument checks shared by the C entry points of the attention
// operators (host code only).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

#include "../../include/kda.h"
#include "kda_internal.h"

namespace kda {
namespace api {

inline kda_status fail(kda_status s, const char* msg) {
    kda::set_last_error(msg);
    return s;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 4096;   // row indices and tile ends stay in 32 bits

inline kda_status launched(hipError_t e, const char* what) {
    if (e == hipSuccess) return KDA_OK;
    kda::set_last_error(std::string(what) + ": " + hipGetErrorString(e));
    return KDA_ERR_HIP;
}

inline bool dtype_ok(int32_t d) { return d == KDA_DTYPE_F32 || d == KDA_DTYPE_BF16; }
inline int elem_size(int32_t d) { return d == KDA_DTYPE_BF16 ? 2 : 4; }

// a stride in elements that keeps 16-byte alignment
inline bool stride_ok(int64_t s, int32_t dtype) { return s * elem_size(dtype) % 16 == 0 && s >= 0 && s < ((int64_t)1 << 40); }

}  // namespace api
}  // namespace kda
