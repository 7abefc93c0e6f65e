// Host side of the entry points on labels and codebooks inside a model
// (include/kmeans.h, last part): argument checks, workspace plans, launches.
// Every check happens before the first enqueue; nothing here allocates device
// memory or synchronizes the stream.
#include "host.h"
#include "rows.h"

using namespace km;

namespace {

constexpr int64_t kMaxB = 65535;
constexpr int64_t kMaxInt = 0x7fffffff;
constexpr int64_t kMaxV = (int64_t)1 << 30;
constexpr int64_t kMaxSide = (int64_t)1 << 20;  // rows or columns of a 4-bit matrix
// Rows of a 4-bit product: its token tiles go in the grid's second axis (65535
// at most).  Tiles of 16 tokens are taken for 2^16 rows or less, whatever the
// matrices, so there are never more than 2^20 / 32 + kRouteMaxE + 1 of them.
constexpr int64_t kMaxTokens = (int64_t)1 << 20;

km_status check_dtype(int xt) {
    if (xt != KM_F32 && xt != KM_F16 && xt != KM_BF16) return fail(KM_EUNSUPPORTED, "unknown dtype %d", xt);
    return KM_OK;
}

// n rows of d elements: non-negative, below 2^31 rows, and of fewer 16-byte
// chunks (8 TB) than the kernels' index arithmetic allows for.
km_status check_rows(int64_t n, int64_t d, int xt, const char* what) {
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

km_status check_table(int64_t B, int64_t N, int64_t V, int64_t d, int xt) {
    if (B < 0 || N < 0) return fail(KM_EINVAL, "negative size: B=%lld N=%lld", (long long)B, (long long)N);
    if (V < 1) return fail(KM_EINVAL, "V must be >= 1 (V=%lld)", (long long)V);
    if (B > kMaxB) return fail(KM_EUNSUPPORTED, "B=%lld > %lld is not supported", (long long)B, (long long)kMaxB);
    if (N > kMaxInt) return fail(KM_EUNSUPPORTED, "N=%lld >= 2^31 is not supported", (long long)N);
    if (V > kMaxV) return fail(KM_EUNSUPPORTED, "V=%lld > 2^30 is not supported", (long long)V);
    KM_TRY(check_rows(B * N, d, xt, "rows"));
    return check_rows(V, d, xt, "table rows");
}

km_status check_route(int64_t T, int64_t top) {
    if (T < 0) return fail(KM_EINVAL, "negative number of tokens: %lld", (long long)T);
    if (top < 1) return fail(KM_EINVAL, "top must be >= 1 (top=%lld)", (long long)top);
    if (T > kMaxInt || top > kMaxInt || T * top > kMaxInt)
        return fail(KM_EUNSUPPORTED, "T*top >= 2^31 is not supported (T=%lld top=%lld)", (long long)T, (long long)top);
    return KM_OK;
}

km_status check_experts(int64_t E) {
    if (E < 1) return fail(KM_EINVAL, "E must be >= 1 (E=%lld)", (long long)E);
    if (E > kRouteMaxE) return fail(KM_EUNSUPPORTED, "E=%lld > %lld is not supported", (long long)E, (long long)kRouteMaxE);
    return KM_OK;
}

struct DispatchPlan {
    size_t hist = 0, prefix = 0, counts = 0, total = 0;
};

DispatchPlan plan_dispatch(int64_t T, int64_t top, int64_t E) {
    DispatchPlan p;
    const int64_t M = T * top;
    if (dispatch_small(T, top)) return p;
    const size_t rows = align_up((size_t)rank_chunks(1, M) * E * sizeof(int32_t));
    p.prefix = rows;
    p.counts = 2 * rows;
    p.total = p.counts + align_up((size_t)E * sizeof(int32_t));
    return p;
}

km_status check_matrix(int64_t M, int64_t K) {
    if (M < 1 || K < 1) return fail(KM_EINVAL, "M and K must be >= 1 (M=%lld K=%lld)", (long long)M, (long long)K);
    if (M > kMaxSide || K > kMaxSide)
        return fail(KM_EUNSUPPORTED, "M=%lld K=%lld: more than 2^20 is not supported", (long long)M, (long long)K);
    return KM_OK;
}

km_status check_codes(int64_t S, int64_t E, int64_t M, int64_t K, int xt) {
    if (S < 0) return fail(KM_EINVAL, "negative number of rows: %lld", (long long)S);
    KM_TRY(check_experts(E));
    KM_TRY(check_matrix(M, K));
    KM_TRY(check_dtype(xt));
    if (xt == KM_F32) return fail(KM_EUNSUPPORTED, "products with 4-bit weights take 16-bit rows, not float32");
    if (S > kMaxTokens) return fail(KM_EUNSUPPORTED, "S=%lld > 2^20 is not supported", (long long)S);
    return KM_OK;
}

km_status run_codes(bool grad, const void* x, int xt, int64_t S, const void* codes, const void* table,
                    int64_t table_rows, const void* scales, int64_t group, int64_t E, int64_t M, int64_t K,
                    const int32_t* offsets, void* out, void* workspace, size_t workspace_bytes, km_stream stream) {
    KM_TRY(check_codes(S, E, M, K, xt));
    if (table_rows != 1 && table_rows != M)
        return fail(KM_EINVAL, "table_rows must be 1 or M (table_rows=%lld M=%lld)", (long long)table_rows, (long long)M);
    if (scales && group != 32 && group != 64 && (group < 128 || group % 128 != 0))
        return fail(group < 1 ? KM_EINVAL : KM_EUNSUPPORTED, "group=%lld: 32, 64 or a multiple of 128 is supported",
                    (long long)group);
    KM_TRY(need(x, S, "x"));
    KM_TRY(need(codes, S, "codes"));
    KM_TRY(need(table, S, "table"));
    KM_TRY(need(out, S, "out"));
    if (E > 1) KM_TRY(need(offsets, S, "offsets"));
    if ((uintptr_t)codes % 16 != 0) return fail(KM_EINVAL, "codes must be 16-byte aligned");
    if (grad) KM_TRY(check_ws_bytes(codes_product_grad_scratch(S, E, M, K), workspace, workspace_bytes));
    const CodesArgs a{x, codes, table, scales, offsets, out, S, E, M, K, group, table_rows};
    const DType t = (DType)xt;
    if (grad) KM_HIP(launch_codes_product_grad(t, a, workspace, (hipStream_t)stream), "codes_product_grad");
    else KM_HIP(launch_codes_product(t, a, (hipStream_t)stream), "codes_product");
    return KM_OK;
}

}  // namespace

extern "C" {

km_status kmeans_lookup(const void* table, km_dtype xt_, int64_t B, int64_t V, int64_t d, const int32_t* labels,
                        int64_t N, float scale, void* out, km_stream stream) {
    const int xt = enum_code(xt_);
    KM_TRY(check_table(B, N, V, d, xt));
    KM_TRY(need(table, B * N, "table"));
    KM_TRY(need(labels, B * N, "labels"));
    KM_TRY(need(out, B * N, "out"));
    KM_HIP(launch_lookup((DType)xt, table, B, V, d, labels, N, scale, out, (hipStream_t)stream), "lookup");
    return KM_OK;
}

size_t kmeans_lookup_grad_workspace_bytes(int64_t B, int64_t N, int64_t d, int64_t V, km_dtype xt_) {
    const int xt = enum_code(xt_);
    if (check_table(B, N, V, d, xt) != KM_OK) return 0;
    return plan_lookup_grad(B, N, d, V, (DType)xt).total;
}

km_status kmeans_lookup_grad(const void* grad, km_dtype xt_, int64_t B, int64_t N, int64_t d, const int32_t* labels,
                             int64_t V, float scale, void* grad_table, km_dtype gt_, void* workspace,
                             size_t workspace_bytes, km_stream stream) {
    const int xt = enum_code(xt_), gt = enum_code(gt_);
    KM_TRY(check_table(B, N, V, d, xt));
    KM_TRY(check_dtype(gt));
    if (gt != xt && gt != KM_F32) return fail(KM_EUNSUPPORTED, "the table's gradient has the rows' dtype or float32");
    KM_TRY(need(grad, B * N, "grad"));
    KM_TRY(need(labels, B * N, "labels"));
    KM_TRY(need(grad_table, B, "grad_table"));
    const LookupGradPlan p = plan_lookup_grad(B, N, d, V, (DType)xt);
    KM_TRY(check_ws_bytes(p.total, workspace, workspace_bytes));
    KM_HIP(launch_lookup_grad((DType)xt, grad, B, N, d, labels, V, scale, (DType)gt, grad_table, p, (char*)workspace,
                              (hipStream_t)stream),
           "lookup_grad");
    return KM_OK;
}

size_t kmeans_dispatch_workspace_bytes(int64_t T, int64_t top, int64_t E) {
    if (check_route(T, top) != KM_OK || check_experts(E) != KM_OK) return 0;
    return plan_dispatch(T, top, E).total;
}

km_status kmeans_dispatch(const void* x, km_dtype xt_, int64_t T, int64_t d, const int32_t* experts, int64_t top,
                          int64_t E, void* rows, int32_t* offsets, int32_t* slots, int32_t* order, void* workspace,
                          size_t workspace_bytes, km_stream stream) {
    const int xt = enum_code(xt_);
    KM_TRY(check_route(T, top));
    KM_TRY(check_experts(E));
    KM_TRY(check_rows(T * top, d, xt, "sorted rows"));
    KM_TRY(need(x, T, "x"));
    KM_TRY(need(experts, T, "experts"));
    KM_TRY(need(rows, T, "rows"));
    KM_TRY(need(offsets, 1, "offsets"));
    KM_TRY(need(slots, T, "slots"));
    KM_TRY(need(order, T, "order"));
    const int64_t M = T * top;
    const DispatchPlan p = plan_dispatch(T, top, E);
    KM_TRY(check_ws_bytes(p.total, workspace, workspace_bytes));
    hipStream_t s = (hipStream_t)stream;
    if (dispatch_small(T, top)) {
        KM_HIP(launch_dispatch_small((DType)xt, x, T, d, top, experts, E, rows, offsets, slots, order, s), "dispatch");
        return KM_OK;
    }
    KM_HIP(launch_route(experts, M, E, at<int32_t>(workspace, p.hist), at<int32_t>(workspace, p.prefix),
                        at<int32_t>(workspace, p.counts), offsets, slots, order, s),
           "route");
    KM_HIP(launch_dispatch_rows((DType)xt, x, T, d, top, slots, offsets + E, rows, order, s), "dispatch");
    return KM_OK;
}

km_status kmeans_combine(const void* rows, km_dtype xt_, int64_t T, int64_t d, int64_t top, const int32_t* slots,
                         const float* weights, void* out, km_stream stream) {
    const int xt = enum_code(xt_);
    KM_TRY(check_route(T, top));
    KM_TRY(check_rows(T * top, d, xt, "sorted rows"));
    KM_TRY(need(rows, T, "rows"));
    KM_TRY(need(slots, T, "slots"));
    KM_TRY(need(out, T, "out"));
    KM_HIP(launch_combine((DType)xt, rows, T, d, top, slots, weights, out, (hipStream_t)stream), "combine");
    return KM_OK;
}

km_status kmeans_combine_grad(const void* grad, const void* rows, km_dtype xt_, int64_t T, int64_t d, int64_t top,
                              const int32_t* slots, const int32_t* order, const float* weights, void* grad_rows,
                              float* grad_weights, km_stream stream) {
    const int xt = enum_code(xt_);
    KM_TRY(check_route(T, top));
    KM_TRY(check_rows(T * top, d, xt, "sorted rows"));
    KM_TRY(need(grad, T, "grad"));
    KM_TRY(need(rows, T, "rows"));
    KM_TRY(need(slots, T, "slots"));
    KM_TRY(need(order, T, "order"));
    KM_TRY(need(weights, T, "weights"));
    KM_TRY(need(grad_rows, T, "grad_rows"));
    KM_TRY(need(grad_weights, T, "grad_weights"));
    KM_HIP(launch_combine_grad((DType)xt, grad, rows, T, d, top, slots, order, weights, grad_rows, grad_weights,
                               (hipStream_t)stream),
           "combine_grad");
    return KM_OK;
}

size_t kmeans_codes_bytes(int64_t M, int64_t K) {
    if (check_matrix(M, K) != KM_OK) return 0;
    return (size_t)code_tiles_m(M) * code_tiles_k(K) * kCodeTile;
}

km_status kmeans_pack_codes(const int32_t* labels, int64_t M, int64_t K, void* codes, km_stream stream) {
    KM_TRY(check_matrix(M, K));
    KM_TRY(need(labels, 1, "labels"));
    KM_TRY(need(codes, 1, "codes"));
    if ((uintptr_t)codes % 16 != 0) return fail(KM_EINVAL, "codes must be 16-byte aligned");
    KM_HIP(launch_pack_codes(labels, M, K, codes, (hipStream_t)stream), "pack_codes");
    return KM_OK;
}

size_t kmeans_codes_workspace_bytes(int64_t S, int64_t E, int64_t M, int64_t K, km_dtype xt_) {
    if (check_codes(S, E, M, K, enum_code(xt_)) != KM_OK) return 0;
    return codes_product_grad_scratch(S, E, M, K);
}

km_status kmeans_codes_product(const void* x, km_dtype xt, int64_t S, const void* codes, const void* table,
                               int64_t table_rows, const void* scales, int64_t group, int64_t E, int64_t M, int64_t K,
                               const int32_t* offsets, void* out, void* workspace, size_t workspace_bytes,
                               km_stream stream) {
    return run_codes(false, x, enum_code(xt), S, codes, table, table_rows, scales, group, E, M, K, offsets, out, workspace,
                     workspace_bytes, stream);
}

km_status kmeans_codes_product_grad(const void* grad, km_dtype xt, int64_t S, const void* codes, const void* table,
                                    int64_t table_rows, const void* scales, int64_t group, int64_t E, int64_t M,
                                    int64_t K, const int32_t* offsets, void* out, void* workspace,
                                    size_t workspace_bytes, km_stream stream) {
    return run_codes(true, grad, enum_code(xt), S, codes, table, table_rows, scales, group, E, M, K, offsets, out, workspace,
                     workspace_bytes, stream);
}

}  // extern "C"
