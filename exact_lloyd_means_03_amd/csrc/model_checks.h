// Checks of sizes and types that the entry points of the operators inside a
// model share (model_api.hip, layer_api.hip).
#pragma once

#include "host.h"
#include "rows.h"

namespace km {

constexpr int64_t kMaxB = 65535;
constexpr int64_t kMaxInt = 0x7fffffff;
constexpr int64_t kMaxV = (int64_t)1 << 30;
constexpr int64_t kMaxSide = (int64_t)1 << 20;  // rows or columns of a 4-bit matrix
// Rows of a 4-bit product: its token tiles go in the grid's second axis (65535
// at most).  Tiles of 16 tokens are taken for 2^16 rows or less, whatever the
// matrices, so there are never more than 2^20 / 32 + kRouteMaxE + 1 of them.
constexpr int64_t kMaxTokens = (int64_t)1 << 20;

inline km_status check_dtype(int xt) {
    if (xt != KM_F32 && xt != KM_F16 && xt != KM_BF16) return fail(KM_EUNSUPPORTED, "unknown dtype %d", xt);
    return KM_OK;
}

// n rows of d elements: non-negative, below 2^31 rows, and of fewer 16-byte
// chunks (8 TB) than the kernels' index arithmetic allows for.
inline km_status check_rows(int64_t n, int64_t d, int xt, const char* what) {
    KM_TRY(check_dtype(xt));
    if (n < 0) return fail(KM_EINVAL, "negative number of %s: %lld", what, (long long)n);
    if (d < 1) return fail(KM_EINVAL, "d must be >= 1 (d=%lld)", (long long)d);
    if (n > kMaxInt) return fail(KM_EUNSUPPORTED, "%lld %s: 2^31 or more are not supported", (long long)n, what);
    if (d > kMaxInt / 16) return fail(KM_EUNSUPPORTED, "d=%lld is not supported", (long long)d);
    const int64_t chunks = row_chunks(d, dtype_bytes((DType)xt));
    if (n * chunks > (int64_t)kMaxInt * 256)
        return fail(KM_EUNSUPPORTED, "%lld %s of %lld elements are not supported in one call", (long long)n, what,
                    (long long)d);
    return KM_OK;
}

inline km_status check_table(int64_t B, int64_t N, int64_t V, int64_t d, int xt) {
    if (B < 0 || N < 0) return fail(KM_EINVAL, "negative size: B=%lld N=%lld", (long long)B, (long long)N);
    if (V < 1) return fail(KM_EINVAL, "V must be >= 1 (V=%lld)", (long long)V);
    if (B > kMaxB) return fail(KM_EUNSUPPORTED, "B=%lld > %lld is not supported", (long long)B, (long long)kMaxB);
    if (N > kMaxInt) return fail(KM_EUNSUPPORTED, "N=%lld >= 2^31 is not supported", (long long)N);
    if (V > kMaxV) return fail(KM_EUNSUPPORTED, "V=%lld > 2^30 is not supported", (long long)V);
    KM_TRY(check_rows(B * N, d, xt, "rows"));
    return check_rows(V, d, xt, "table rows");
}

inline km_status check_route(int64_t T, int64_t top) {
    if (T < 0) return fail(KM_EINVAL, "negative number of tokens: %lld", (long long)T);
    if (top < 1) return fail(KM_EINVAL, "top must be >= 1 (top=%lld)", (long long)top);
    if (T > kMaxInt || top > kMaxInt || T * top > kMaxInt)
        return fail(KM_EUNSUPPORTED, "T*top >= 2^31 is not supported (T=%lld top=%lld)", (long long)T, (long long)top);
    return KM_OK;
}

inline km_status check_experts(int64_t E) {
    if (E < 1) return fail(KM_EINVAL, "E must be >= 1 (E=%lld)", (long long)E);
    if (E > kRouteMaxE) return fail(KM_EUNSUPPORTED, "E=%lld > %lld is not supported", (long long)E, (long long)kRouteMaxE);
    return KM_OK;
}

inline km_status check_matrix(int64_t M, int64_t K) {
    if (M < 1 || K < 1) return fail(KM_EINVAL, "M and K must be >= 1 (M=%lld K=%lld)", (long long)M, (long long)K);
    if (M > kMaxSide || K > kMaxSide)
        return fail(KM_EUNSUPPORTED, "M=%lld K=%lld: more than 2^20 is not supported", (long long)M, (long long)K);
    return KM_OK;
}

}  // namespace km
