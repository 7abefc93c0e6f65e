// Host-side helpers shared by the files that hold C ABI entry points:
// status reporting, argument checks and workspace carving.
#pragma once

#include <stdint.h>
#include <string.h>

#include "../../include/kmeans.h"
#include "common.h"

namespace km {

// Records the message of kmeans_last_error() and returns st.
km_status fail(km_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
km_status hip_fail(hipError_t e, const char* where);

inline size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

// The code of an enum argument as the caller passed it: a C caller may pass
// any int, and reading a value outside the enumerators through the enum type
// is undefined, so the bytes are read as an int.
template <typename E>
inline int enum_code(const E& e) {
    static_assert(sizeof(E) == sizeof(int), "enums of the ABI are int-sized");
    int v;
    memcpy(&v, &e, sizeof v);
    return v;
}

inline km_status need(const void* p, int64_t n, const char* name) {
    if (n > 0 && p == nullptr) return fail(KM_EINVAL, "%s is NULL", name);
    return KM_OK;
}

inline km_status check_ws_bytes(size_t total, const void* ws, size_t bytes) {
    if (total == 0) return KM_OK;
    if (ws == nullptr) return fail(KM_EINVAL, "workspace is NULL (%zu bytes needed)", total);
    if ((uintptr_t)ws % 256 != 0) return fail(KM_EINVAL, "workspace must be 256-byte aligned");
    if (bytes < total)
        return fail(KM_EWORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", bytes, total);
    return KM_OK;
}

#define KM_TRY(expr)                       \
    do {                                   \
        km_status _st = (expr);            \
        if (_st != KM_OK) return _st;      \
    } while (0)

#define KM_HIP(expr, where)                               \
    do {                                                  \
        hipError_t _e = (expr);                           \
        if (_e != hipSuccess) return hip_fail(_e, where); \
    } while (0)

template <typename P>
inline P* at(void* ws, size_t off) {
    return (P*)((char*)ws + off);
}

}  // namespace km
