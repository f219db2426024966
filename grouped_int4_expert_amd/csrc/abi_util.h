// Host-side helpers of the C ABI: limits, alignment and overlap checks, and
// workspace carving.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmoe.h"

namespace qmoe {

constexpr int MAX_EXPERTS = 1024;
constexpr int MAX_TOPK = 64;

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int64_t align256(int64_t v) { return (v + 255) & ~int64_t(255); }

inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    if (!a || !b || na <= 0 || nb <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? QMOE_OK : QMOE_ERR_HIP; }

// Workspace carving with 256-byte alignment.
struct Carver {
    char *base;
    int64_t off = 0;
    explicit Carver(void *b) : base(static_cast<char *>(b)) {}
    template <typename T>
    T *take(int64_t count) {
        T *p = base ? reinterpret_cast<T *>(base + off) : nullptr;
        off = align256(off + count * (int64_t)sizeof(T));
        return p;
    }
};

}  // namespace qmoe
