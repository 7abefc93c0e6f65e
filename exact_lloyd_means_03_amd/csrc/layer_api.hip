// Host side of the entry points of a layer of 8-bit experts (include/kmeans.h,
// last part): argument checks, workspace plans, launches.  Every check happens
// before the first enqueue; nothing here allocates device memory or
// synchronizes the stream.
#include "host.h"
#include "model_checks.h"
#include "codes8.h"

using namespace km;

namespace {

km_status check_norm(int64_t T, int64_t d, int xt, int wt, const void* weight, float eps) {
    KM_TRY(check_rows(T, d, xt, "rows"));
    if (!norm_fits(d, (DType)xt)) return fail(KM_EUNSUPPORTED, "d=%lld: rows of more than 64 KB are not supported", (long long)d);
    if (weight) {
        KM_TRY(check_dtype(wt));
        if (wt != xt && wt != KM_F32) return fail(KM_EUNSUPPORTED, "the weight has the rows' dtype or float32");
    }
    if (!(eps >= 0.f)) return fail(KM_EINVAL, "eps must be >= 0 (eps=%g)", (double)eps);
    return KM_OK;
}

km_status check_gate(int64_t T, int64_t E, int64_t top) {
    if (T < 0) return fail(KM_EINVAL, "negative number of tokens: %lld", (long long)T);
    KM_TRY(check_experts(E));
    if (top < 1 || top > E) return fail(KM_EINVAL, "top must be in 1 .. E (top=%lld E=%lld)", (long long)top, (long long)E);
    if (!gate_top_fits(top)) return fail(KM_EUNSUPPORTED, "top=%lld > 64 is not supported", (long long)top);
    if (T > kMaxInt || T * top > kMaxInt)
        return fail(KM_EUNSUPPORTED, "T*top >= 2^31 is not supported (T=%lld top=%lld)", (long long)T, (long long)top);
    return KM_OK;
}

km_status check_block(int64_t S, int64_t E, int64_t M, int64_t K) {
    if (S < 0) return fail(KM_EINVAL, "negative number of rows: %lld", (long long)S);
    KM_TRY(check_experts(E));
    KM_TRY(check_matrix(M, K));
    if (S > kMaxTokens) return fail(KM_EUNSUPPORTED, "S=%lld > 2^20 is not supported", (long long)S);
    return KM_OK;
}

km_status run_block(bool grad, const void* x, const float* x_scales, int64_t S, const void* codes, const float* scales,
                    int64_t E, int64_t M, int64_t K, const int32_t* offsets, const int32_t* order, int64_t top,
                    void* out, int ot, void* workspace, size_t workspace_bytes, km_stream stream) {
    KM_TRY(check_block(S, E, M, K));
    KM_TRY(check_dtype(ot));
    KM_TRY(need(x, S, grad ? "grad" : "x"));
    KM_TRY(need(x_scales, S, grad ? "grad_scales" : "x_scales"));
    KM_TRY(need(codes, S, "codes"));
    KM_TRY(need(scales, S, "scales"));
    KM_TRY(need(out, S, "out"));
    if (E > 1) KM_TRY(need(offsets, S, "offsets"));
    if (order && (top < 1 || S % top != 0))
        return fail(KM_EINVAL, "S must be a multiple of top with an order (S=%lld top=%lld)", (long long)S, (long long)top);
    const size_t n = grad ? block_product_grad_scratch(S, E, M, K) : block_product_scratch(S, E, M, K);
    KM_TRY(check_ws_bytes(n, workspace, workspace_bytes));
    const BlockArgs a{x, x_scales, codes, scales, offsets, order, out, S, E, M, K, top};
    KM_HIP(launch_block_product((DType)ot, grad, a, workspace, (hipStream_t)stream),
           grad ? "block_product_grad" : "block_product");
    return KM_OK;
}

}  // namespace

extern "C" {

km_status kmeans_quantize(const void* x, km_dtype xt_, int64_t B, int64_t M, int64_t K, int64_t rows, void* codes,
                          float* scales, km_stream stream) {
    const int xt = enum_code(xt_);
    KM_TRY(check_dtype(xt));
    if (rows != 1 && rows != kBlock8) return fail(KM_EINVAL, "rows must be 1 or 128 (rows=%lld)", (long long)rows);
    if (B < 0 || M < 0) return fail(KM_EINVAL, "negative size: B=%lld M=%lld", (long long)B, (long long)M);
    if (K < 1) return fail(KM_EINVAL, "K must be >= 1 (K=%lld)", (long long)K);
    if (B > kMaxB) return fail(KM_EUNSUPPORTED, "B=%lld > %lld is not supported", (long long)B, (long long)kMaxB);
    if (K > kMaxSide || (rows != 1 && M > kMaxSide))
        return fail(KM_EUNSUPPORTED, "M=%lld K=%lld: more than 2^20 is not supported", (long long)M, (long long)K);
    if (M > kMaxInt) return fail(KM_EUNSUPPORTED, "M=%lld >= 2^31 is not supported", (long long)M);
    if (rows == 1) KM_TRY(check_rows(B * M, K, xt, "rows"));
    KM_TRY(need(x, B * M, "x"));
    KM_TRY(need(codes, B * M, "codes"));
    KM_TRY(need(scales, B * M, "scales"));
    KM_HIP(launch_quantize((DType)xt, x, B, M, K, rows != 1, codes, scales, (hipStream_t)stream), "quantize");
    return KM_OK;
}

km_status kmeans_norm(const void* x, km_dtype xt_, int64_t T, int64_t d, const void* residual, const void* weight,
                      km_dtype wt_, float eps, void* h, void* y, void* codes, float* scales, km_stream stream) {
    const int xt = enum_code(xt_), wt = enum_code(wt_);
    KM_TRY(check_norm(T, d, xt, wt, weight, eps));
    KM_TRY(need(x, T, "x"));
    if ((codes == nullptr) != (scales == nullptr)) return fail(KM_EINVAL, "codes and scales go together");
    if (T > 0 && (y == nullptr) == (codes == nullptr)) return fail(KM_EINVAL, "exactly one of y and codes must be given");
    KM_HIP(launch_norm((DType)xt, x, T, d, residual, weight, (DType)wt, eps, residual ? h : nullptr, y, codes, scales,
                       (hipStream_t)stream),
           "norm");
    return KM_OK;
}

size_t kmeans_norm_grad_workspace_bytes(int64_t T, int64_t d, km_dtype xt_) {
    const int xt = enum_code(xt_);
    if (check_norm(T, d, xt, xt, nullptr, 0.f) != KM_OK) return 0;
    return norm_grad_scratch(T, d, (DType)xt);
}

km_status kmeans_norm_grad(const void* grad, const void* h, km_dtype xt_, int64_t T, int64_t d, const void* grad_residual,
                           const void* weight, km_dtype wt_, float eps, void* grad_x, void* grad_weight, void* workspace,
                           size_t workspace_bytes, km_stream stream) {
    const int xt = enum_code(xt_), wt = enum_code(wt_);
    KM_TRY(check_norm(T, d, xt, wt, weight ? weight : grad_weight, eps));
    KM_TRY(need(grad, T, "grad"));
    KM_TRY(need(h, T, "h"));
    KM_TRY(need(grad_x, T, "grad_x"));
    if (grad_weight) KM_TRY(check_ws_bytes(norm_grad_scratch(T, d, (DType)xt), workspace, workspace_bytes));
    KM_HIP(launch_norm_grad((DType)xt, grad, h, T, d, grad_residual, weight, (DType)wt, eps, grad_x, grad_weight,
                            workspace, (hipStream_t)stream),
           "norm_grad");
    return KM_OK;
}

size_t kmeans_gate_workspace_bytes(int64_t T, int64_t E) {
    if (check_gate(T, E, 1) != KM_OK) return 0;
    return gate_scratch(T, E);
}

km_status kmeans_gate(const void* logits, km_dtype xt_, int64_t T, int64_t E, int64_t top, int32_t normalize,
                      int32_t* experts, float* weights, int32_t* counts, float* shares, float* loss, void* workspace,
                      size_t workspace_bytes, km_stream stream) {
    const int xt = enum_code(xt_);
    KM_TRY(check_gate(T, E, top));
    KM_TRY(check_dtype(xt));
    KM_TRY(need(logits, T, "logits"));
    KM_TRY(need(experts, T, "experts"));
    KM_TRY(need(weights, T, "weights"));
    KM_TRY(need(counts, 1, "counts"));
    KM_TRY(need(shares, 1, "shares"));
    KM_TRY(need(loss, 1, "loss"));
    KM_TRY(check_ws_bytes(gate_scratch(T, E), workspace, workspace_bytes));
    KM_HIP(launch_gate((DType)xt, logits, T, E, top, normalize != 0, experts, weights, counts, shares, loss, workspace,
                       (hipStream_t)stream),
           "gate");
    return KM_OK;
}

km_status kmeans_gate_grad(const void* logits, km_dtype xt_, int64_t T, int64_t E, int64_t top, int32_t normalize,
                           const int32_t* experts, const int32_t* counts, const float* grad_weights,
                           const float* grad_loss, void* grad_logits, km_stream stream) {
    const int xt = enum_code(xt_);
    KM_TRY(check_gate(T, E, top));
    KM_TRY(check_dtype(xt));
    KM_TRY(need(logits, T, "logits"));
    if (grad_weights) KM_TRY(need(experts, T, "experts"));
    if (grad_loss) KM_TRY(need(counts, T, "counts"));
    KM_TRY(need(grad_logits, T, "grad_logits"));
    KM_HIP(launch_gate_grad((DType)xt, logits, T, E, top, normalize != 0, experts, counts, grad_weights, grad_loss,
                            grad_logits, (hipStream_t)stream),
           "gate_grad");
    return KM_OK;
}

km_status kmeans_block_product(const void* x, const float* x_scales, int64_t S, const void* codes, const float* scales,
                               int64_t E, int64_t M, int64_t K, const int32_t* offsets, const int32_t* order,
                               int64_t top, void* out, km_dtype ot, void* workspace, size_t workspace_bytes,
                               km_stream stream) {
    return run_block(false, x, x_scales, S, codes, scales, E, M, K, offsets, order, top, out, enum_code(ot), workspace,
                     workspace_bytes, stream);
}

size_t kmeans_block_product_workspace_bytes(int64_t S, int64_t E, int64_t M, int64_t K) {
    if (check_block(S, E, M, K) != KM_OK) return 0;
    return block_product_scratch(S, E, M, K);
}

km_status kmeans_block_product_grad(const void* grad, const float* grad_scales, int64_t S, const void* codes,
                                    const float* scales, int64_t E, int64_t M, int64_t K, const int32_t* offsets,
                                    void* out, km_dtype ot, void* workspace, size_t workspace_bytes, km_stream stream) {
    return run_block(true, grad, grad_scales, S, codes, scales, E, M, K, offsets, nullptr, 1, out, enum_code(ot),
                     workspace, workspace_bytes, stream);
}

size_t kmeans_block_product_grad_workspace_bytes(int64_t S, int64_t E, int64_t M, int64_t K) {
    if (check_block(S, E, M, K) != KM_OK) return 0;
    return block_product_grad_scratch(S, E, M, K);
}

}  // extern "C"
