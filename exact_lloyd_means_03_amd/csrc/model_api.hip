// Host side of the entry points on labels and codebooks inside a model
// (include/kmeans.h, last part): argument checks, workspace plans, launches.
// Every check happens before the first enqueue; nothing here allocates device
// memory or synchronizes the stream.
#include "host.h"
#include "model_checks.h"
#include "rows.h"

using namespace km;

namespace {

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

size_t kmeans_plan_workspace_bytes(int64_t T, int64_t top, int64_t E) {
    return kmeans_dispatch_workspace_bytes(T, top, E);
}

km_status kmeans_plan(const int32_t* experts, int64_t T, int64_t top, int64_t E, int32_t* offsets, int32_t* slots,
                      int32_t* order, void* workspace, size_t workspace_bytes, km_stream stream) {
    KM_TRY(check_route(T, top));
    KM_TRY(check_experts(E));
    KM_TRY(need(experts, T, "experts"));
    KM_TRY(need(offsets, 1, "offsets"));
    KM_TRY(need(slots, T, "slots"));
    KM_TRY(need(order, T, "order"));
    const int64_t M = T * top;
    const DispatchPlan p = plan_dispatch(T, top, E);
    KM_TRY(check_ws_bytes(p.total, workspace, workspace_bytes));
    hipStream_t s = (hipStream_t)stream;
    if (dispatch_small(T, top)) {  // (rows of no elements)
        KM_HIP(launch_dispatch_small(DType::F32, nullptr, T, 0, top, experts, E, nullptr, offsets, slots, order, s), "plan");
        return KM_OK;
    }
    KM_HIP(launch_route(experts, M, E, at<int32_t>(workspace, p.hist), at<int32_t>(workspace, p.prefix),
                        at<int32_t>(workspace, p.counts), offsets, slots, order, s),
           "plan");
    KM_HIP(launch_plan_tail(offsets + E, M, order, s), "plan");
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
