// Argument checks and workspace helpers shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "moe.h"

namespace moe {

// the workspace's header: the error flag and internal counters
constexpr size_t kHeaderBytes = 256;

inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

inline int32_t check_ptrs(std::initializer_list<const void*> required) {
    for (const void* p : required)
        if (p == nullptr || !aligned16(p)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

inline int32_t check_opt(std::initializer_list<const void*> optional) {
    for (const void* p : optional)
        if (p != nullptr && !aligned16(p)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

inline int32_t hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

template <typename T>
T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

#define MOE_TRY(expr)                       \
    do {                                    \
        const int32_t _rc = (expr);         \
        if (_rc != MOE_OK) return _rc;      \
    } while (0)

}  // namespace moe
