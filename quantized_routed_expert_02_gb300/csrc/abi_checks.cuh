// Argument checks shared by the files that define entry points.
#pragma once

#include "common.cuh"

namespace moeq4k {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline moe_status check_ptr(const void *p, size_t align) {
    if (p == nullptr) return MOE_ERR_NULL;
    if (!aligned(p, align)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

// A pointer that may be NULL.
inline moe_status check_opt(const void *p, size_t align) {
    return p == nullptr || aligned(p, align) ? MOE_OK : MOE_ERR_MISALIGNED;
}

inline bool finite_f(float v) { return v >= -3.402823466e38f && v <= 3.402823466e38f; }

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace moeq4k

#define MOE_TRY(expr)                        \
    do {                                     \
        moe_status _s = (expr);              \
        if (_s != MOE_OK) return _s;         \
    } while (0)
