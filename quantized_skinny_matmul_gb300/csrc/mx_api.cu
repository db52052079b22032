// mx_api.cu -- the C entry points of the microscaled formats, routing and the experts' products:
// argument checks (nothing is launched before they pass), then the launchers.
#include <cmath>

#include "mx.cuh"

namespace gq {
namespace {

#define GQ_TRY(expr)                       \
    do {                                   \
        gq_status _st = (expr);            \
        if (_st != GQ_OK) return _st;      \
    } while (0)

gq_status check_type(gq_type type, const char *name) {
    if (type != GQ_TYPE_F32 && type != GQ_TYPE_BF16) return fail(GQ_ERR_INVALID_ARG, "%s=%d is no gq_type", name, (int)type);
    return GQ_OK;
}

gq_status check_kind(gq_mx_kind kind) {
    if (kind != GQ_MX_E2M1 && kind != GQ_MX_E4M3) return fail(GQ_ERR_INVALID_ARG, "kind=%d is no gq_mx_kind", (int)kind);
    return GQ_OK;
}

// rows of `type`: each starts on 16 bytes
gq_status check_stride(int64_t ld, int64_t n, gq_type type, const char *name) {
    const int64_t unit = type == GQ_TYPE_BF16 ? 8 : 4;
    if (ld < n || ld % unit != 0 || ld > (1LL << 31))
        return fail(GQ_ERR_INVALID_ARG, "%s=%lld must be a multiple of %lld and at least %lld", name, (long long)ld, (long long)unit,
                    (long long)n);
    return GQ_OK;
}

gq_status check_ptr4(const void *p, const char *name) {
    if (!p) return fail(GQ_ERR_INVALID_ARG, "%s is NULL", name);
    if ((uintptr_t)p & 3u) return fail(GQ_ERR_MISALIGNED, "%s (%p) is not 4-byte aligned", name, p);
    return GQ_OK;
}

// the operands of a product: activations, plan, sizes
gq_status check_product(const void *repacked, const gq_mx_rows *x, const gq_expert_rows *plan, int64_t N, int64_t K,
                        int64_t parts) {
    GQ_TRY(check_sizes(1, N, K));
    if (!x) return fail(GQ_ERR_INVALID_ARG, "x is NULL");
    if (x->rows <= 0 || x->rows >= (1LL << 30)) return fail(GQ_ERR_INVALID_ARG, "x->rows must be in [1, 2^30) (got %lld)", (long long)x->rows);
    int64_t count = parts;
    if (plan) {
        if (plan->E < 1 || plan->E > 1024) return fail(GQ_ERR_INVALID_ARG, "E must be in [1, 1024] (got %lld)", (long long)plan->E);
        if (plan->R < 1 || plan->R >= (1LL << 30)) return fail(GQ_ERR_INVALID_ARG, "R must be in [1, 2^30) (got %lld)", (long long)plan->R);
        if (!plan->rows && x->rows < plan->R)
            return fail(GQ_ERR_INVALID_ARG, "x has %lld rows, the plan %lld", (long long)x->rows, (long long)plan->R);
        GQ_TRY(check_ptr4(plan->offsets, "plan->offsets"));
        if (plan->rows) GQ_TRY(check_ptr4(plan->rows, "plan->rows"));
        count *= plan->E;
    }
    if (!gq_mxfp4_repacked_bytes(count, N, K)) return fail(GQ_ERR_INVALID_ARG, "weights too large");
    GQ_TRY(check_ptr(repacked, "repacked"));
    GQ_TRY(check_ptr(x->codes, "x->codes"));
    return check_ptr(x->scales, "x->scales");
}

}  // namespace
}  // namespace gq

using namespace gq;

extern "C" {

size_t gq_mx_scale_cols(int64_t K) { return K <= 0 || K % QK ? 0 : (size_t)((K + 511) / 512) * 16; }

gq_status gq_quantize_mx(const void *x, int64_t ldx, gq_type type, gq_mx_kind kind, void *codes, uint8_t *scales,
                         int64_t M, int64_t K, cudaStream_t stream) {
    GQ_TRY(check_sizes(M, 1, K));
    GQ_TRY(check_type(type, "type"));
    GQ_TRY(check_kind(kind));
    GQ_TRY(check_stride(ldx, K, type, "ldx"));
    GQ_TRY(check_ptr(x, "x"));
    GQ_TRY(check_ptr(codes, "codes"));
    GQ_TRY(check_ptr(scales, "scales"));
    GQ_TRY(check_device());
    GQ_TRY(launch_quantize_mx(x, ldx, type == GQ_TYPE_BF16, kind == GQ_MX_E2M1, codes, scales, M, K, stream));
    return ok();
}

gq_status gq_dequantize_mx(const void *codes, const uint8_t *scales, gq_mx_kind kind, void *y, gq_type type,
                           int64_t M, int64_t K, cudaStream_t stream) {
    GQ_TRY(check_sizes(M, 1, K));
    GQ_TRY(check_type(type, "type"));
    GQ_TRY(check_kind(kind));
    GQ_TRY(check_ptr(codes, "codes"));
    GQ_TRY(check_ptr(scales, "scales"));
    GQ_TRY(check_ptr(y, "y"));
    GQ_TRY(check_device());
    GQ_TRY(launch_dequantize_mx(codes, scales, kind == GQ_MX_E2M1, y, type == GQ_TYPE_BF16, M, K, stream));
    return ok();
}

gq_status gq_rms_norm_mx(const void *x, int64_t ldx, const void *residual, int64_t ldr, gq_type type,
                         const float *weight, double eps, void *h, int64_t ldh, void *y, gq_type ytype,
                         void *codes, uint8_t *scales, int64_t M, int64_t K, cudaStream_t stream) {
    GQ_TRY(check_sizes(M, 1, K));
    if (K > 32768) return fail(GQ_ERR_INVALID_ARG, "K must be at most 32768 for the norm (got %lld)", (long long)K);
    GQ_TRY(check_type(type, "type"));
    GQ_TRY(check_type(ytype, "ytype"));
    if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(GQ_ERR_INVALID_ARG, "eps must be finite and not negative");
    GQ_TRY(check_stride(ldx, K, type, "ldx"));
    GQ_TRY(check_ptr(x, "x"));
    if (residual) {
        GQ_TRY(check_stride(ldr, K, type, "ldr"));
        GQ_TRY(check_ptr(residual, "residual"));
    }
    if (weight) GQ_TRY(check_ptr(weight, "weight"));
    if (h) {
        GQ_TRY(check_stride(ldh, K, type, "ldh"));
        GQ_TRY(check_ptr(h, "h"));
    }
    if (y) GQ_TRY(check_ptr(y, "y"));
    if (!codes != !scales) return fail(GQ_ERR_INVALID_ARG, "codes and scales go together");
    if (codes) {
        GQ_TRY(check_ptr(codes, "codes"));
        GQ_TRY(check_ptr(scales, "scales"));
    }
    if (!h && !y && !codes) return fail(GQ_ERR_INVALID_ARG, "h, y and codes are all NULL");
    GQ_TRY(check_device());
    GQ_TRY(launch_rms_norm_mx(x, ldx, residual, ldr, type == GQ_TYPE_BF16, weight, eps, h, ldh, y, ytype == GQ_TYPE_BF16, codes,
                              scales, M, K, stream));
    return ok();
}

size_t gq_mxfp4_repacked_bytes(int64_t count, int64_t N, int64_t K) {
    if (count <= 0 || N <= 0 || K <= 0 || K % QK || N > (1LL << 30) || K > (1LL << 30) || count > 2048) return 0;
    const int64_t G = (N + MX_TILE - 1) / MX_TILE, KT = (K + MX_TILE - 1) / MX_TILE;
    // 2^24 tiles are 146 GB; their numbers stay far within 32 bits
    if (G * KT > (1LL << 24) || count * G * KT >= (1LL << 24)) return 0;
    return (size_t)(count * G * KT) * (MX_TILE_CODES + MX_TILE_SCALES);
}

gq_status gq_repack_mxfp4(const void *codes, const uint8_t *scales, void *repacked, int64_t count, int64_t N,
                          int64_t K, cudaStream_t stream) {
    GQ_TRY(check_sizes(1, N, K));
    const size_t bytes = gq_mxfp4_repacked_bytes(count, N, K);
    if (!bytes)
        return fail(GQ_ERR_INVALID_ARG, "count=%lld matrices of %lld x %lld: out of range", (long long)count, (long long)N, (long long)K);
    GQ_TRY(check_ptr(codes, "codes"));
    GQ_TRY(check_ptr(scales, "scales"));
    GQ_TRY(check_ptr(repacked, "repacked"));
    const uintptr_t r = (uintptr_t)repacked, c = (uintptr_t)codes, sc = (uintptr_t)scales;
    if ((c < r + bytes && r < c + (size_t)count * N * K / 2) || (sc < r + bytes && r < sc + (size_t)count * N * gq_mx_scale_cols(K)))
        return fail(GQ_ERR_INVALID_ARG, "repacked overlaps its inputs");
    GQ_TRY(check_device());
    GQ_TRY(launch_repack_mxfp4(codes, scales, repacked, count, N, K, stream));
    return ok();
}

gq_status gq_mul_mat_mxfp4_mx(const void *repacked, const gq_mx_rows *x, const gq_expert_rows *plan, void *dst,
                              int64_t ldd, gq_type type, int64_t N, int64_t K, cudaStream_t stream) {
    GQ_TRY(check_product(repacked, x, plan, N, K, 1));
    GQ_TRY(check_type(type, "type"));
    if (ldd < N || ldd > (1LL << 31)) return fail(GQ_ERR_INVALID_ARG, "ldd=%lld must be at least N=%lld", (long long)ldd, (long long)N);
    GQ_TRY(check_ptr(dst, "dst"));
    GQ_TRY(check_device());
    GQ_TRY(launch_mx_product(repacked, *x, plan, dst, ldd, type == GQ_TYPE_BF16, nullptr, nullptr, N, K, stream));
    return ok();
}

gq_status gq_mul_mat_mxfp4(const void *repacked, const void *x, int64_t ldx, gq_type xtype, void *dst, int64_t ldd,
                           gq_type type, int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
    GQ_TRY(check_sizes(M, N, K));
    GQ_TRY(check_type(xtype, "xtype"));
    GQ_TRY(check_type(type, "type"));
    GQ_TRY(check_stride(ldx, K, xtype, "ldx"));
    if (M >= (1LL << 30) || !gq_mxfp4_repacked_bytes(1, N, K))
        return fail(GQ_ERR_INVALID_ARG, "sizes too large (M=%lld N=%lld K=%lld)", (long long)M, (long long)N, (long long)K);
    if (ldd < N || ldd > (1LL << 31)) return fail(GQ_ERR_INVALID_ARG, "ldd=%lld must be at least N=%lld", (long long)ldd, (long long)N);
    GQ_TRY(check_ptr(repacked, "repacked"));
    GQ_TRY(check_ptr(x, "x"));
    GQ_TRY(check_ptr(dst, "dst"));
    GQ_TRY(check_device());
    if (M <= MX_FEW_ROWS) {
        GQ_TRY(launch_mx_product_few(repacked, x, ldx, xtype == GQ_TYPE_BF16, dst, ldd, type == GQ_TYPE_BF16, M, N, K, stream));
        return ok();
    }
    Workspace ws;
    const size_t scales = (size_t)M * gq_mx_scale_cols(K);
    GQ_TRY(get_workspace(stream, 0, scales + (size_t)M * K, &ws));
    GQ_TRY(launch_quantize_mx(x, ldx, xtype == GQ_TYPE_BF16, false, ws.data + scales, ws.data, M, K, stream));
    const gq_mx_rows rows{M, ws.data + scales, ws.data};
    GQ_TRY(launch_mx_product(repacked, rows, nullptr, dst, ldd, type == GQ_TYPE_BF16, nullptr, nullptr, N, K, stream));
    return ok();
}

gq_status gq_swiglu_mxfp4_mx(const void *repacked, const gq_mx_rows *x, const gq_expert_rows *plan, void *codes,
                             uint8_t *scales, int64_t F, int64_t K, cudaStream_t stream) {
    GQ_TRY(check_product(repacked, x, plan, F, K, 2));
    if (F % QK) return fail(GQ_ERR_INVALID_ARG, "F=%lld is not a multiple of 32", (long long)F);
    GQ_TRY(check_ptr(codes, "codes"));
    GQ_TRY(check_ptr(scales, "scales"));
    GQ_TRY(check_device());
    GQ_TRY(launch_mx_product(repacked, *x, plan, nullptr, 0, false, codes, scales, F, K, stream));
    return ok();
}

gq_status gq_route(const gq_router *router, const void *logits, int64_t ldl, gq_type type, const int32_t *used,
                   int32_t *ids, float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, int64_t T,
                   cudaStream_t stream) {
    if (!router) return fail(GQ_ERR_INVALID_ARG, "router is NULL");
    const gq_router &r = *router;
    if (r.E < 1 || r.E > 1024) return fail(GQ_ERR_INVALID_ARG, "E must be in [1, 1024] (got %lld)", (long long)r.E);
    if (r.score != GQ_SCORE_SOFTMAX && r.score != GQ_SCORE_SIGMOID)
        return fail(GQ_ERR_INVALID_ARG, "score=%lld is no gq_score", (long long)r.score);
    if (r.groups < 1 || r.groups > 32 || r.E % r.groups || r.top_groups < 1 || r.top_groups > r.groups)
        return fail(GQ_ERR_INVALID_ARG, "need 1 to 32 groups that divide E=%lld, and top_groups of them (got %lld, %lld)", (long long)r.E,
                    (long long)r.groups, (long long)r.top_groups);
    if (r.group_best != 1 && r.group_best != 2)
        return fail(GQ_ERR_INVALID_ARG, "group_best must be 1 or 2 (got %lld)", (long long)r.group_best);
    if (r.top_k < 1 || r.top_k > 32 || r.top_k > r.top_groups * (r.E / r.groups))
        return fail(GQ_ERR_INVALID_ARG, "top_k must be in [1, 32] and at most the %lld experts that can be chosen (got %lld)",
                    (long long)(r.top_groups * (r.E / r.groups)), (long long)r.top_k);
    if (!std::isfinite(r.factor)) return fail(GQ_ERR_INVALID_ARG, "factor is not finite");
    GQ_TRY(check_type(type, "type"));
    if (T <= 0 || T >= (1LL << 30) || T * r.top_k >= (1LL << 30))
        return fail(GQ_ERR_INVALID_ARG, "T must be positive, T * top_k below 2^30 (got %lld)", (long long)T);
    if (ldl < r.E || ldl > (1LL << 31)) return fail(GQ_ERR_INVALID_ARG, "ldl=%lld must be at least E=%lld", (long long)ldl, (long long)r.E);
    GQ_TRY(check_ptr(logits, "logits"));
    if (r.bias) GQ_TRY(check_ptr(r.bias, "bias"));
    if (used) GQ_TRY(check_ptr4(used, "used"));
    GQ_TRY(check_ptr(ids, "ids"));
    GQ_TRY(check_ptr(weights, "weights"));
    if (offsets || rows || pos) {
        GQ_TRY(check_ptr(offsets, "offsets"));
        GQ_TRY(check_ptr(rows, "rows"));
        GQ_TRY(check_ptr(pos, "pos"));
    }
    GQ_TRY(check_device());
    GQ_TRY(launch_route(r, logits, ldl, type == GQ_TYPE_BF16, used, ids, weights, offsets, rows, pos, T, stream));
    return ok();
}

gq_status gq_experts_combine(const float *y, int64_t R, const int32_t *pos, const float *weights, int64_t top_k,
                             const void *residual, int64_t ldr, gq_type rtype, void *out, int64_t ldo, gq_type type,
                             int64_t T, int64_t N, cudaStream_t stream) {
    if (T <= 0 || N <= 0 || N % 8 || T >= (1LL << 30) || N > (1LL << 30))
        return fail(GQ_ERR_INVALID_ARG, "T and N must be positive, N a multiple of 8 (T=%lld N=%lld)", (long long)T, (long long)N);
    if (R <= 0 || R >= (1LL << 30)) return fail(GQ_ERR_INVALID_ARG, "R must be in [1, 2^30) (got %lld)", (long long)R);
    if (top_k < 1 || top_k > 32) return fail(GQ_ERR_INVALID_ARG, "top_k must be in [1, 32] (got %lld)", (long long)top_k);
    GQ_TRY(check_type(type, "type"));
    GQ_TRY(check_ptr(y, "y"));
    GQ_TRY(check_ptr(pos, "pos"));
    GQ_TRY(check_ptr(weights, "weights"));
    if (residual) {
        GQ_TRY(check_type(rtype, "rtype"));
        GQ_TRY(check_stride(ldr, N, rtype, "ldr"));
        GQ_TRY(check_ptr(residual, "residual"));
    }
    GQ_TRY(check_stride(ldo, N, type, "ldo"));
    GQ_TRY(check_ptr(out, "out"));
    GQ_TRY(check_device());
    GQ_TRY(launch_experts_combine(y, R, pos, weights, top_k, residual, ldr, residual && rtype == GQ_TYPE_BF16, out, ldo,
                                  type == GQ_TYPE_BF16, T, N, stream));
    return ok();
}

}  // extern "C"
