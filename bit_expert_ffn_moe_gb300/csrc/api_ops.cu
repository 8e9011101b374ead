// api_ops.cu -- extern "C" entry points beside the layer (include/moe.h): routing rules and their gradient, the
// weighted sum's gradients, dense NVFP4 products.  Argument checks and launches; nothing allocates device
// memory and nothing throws past these functions.
#include <math.h>

#include "ops.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Whether all of these (null ones among them) start on 4 bytes: arrays of floats and of ints.
template <typename... P>
bool words(const P*... p) { return (aligned(p, 4) && ...); }

#define MOE_TRY(expr)                \
    do {                             \
        moe_status _s = (expr);      \
        if (_s != MOE_OK) return _s; \
    } while (0)

// Launches may allocate host memory (tables of the runtime and of launch.cu): no exception leaves a C entry.
template <typename F>
moe_status launch(F f) {
    try {
        MOE_TRY(check_device());
        return from_cuda(f());
    } catch (...) {
        return from_cuda(cudaErrorMemoryAllocation);
    }
}

size_t dtype_size(moe_dtype t) { return t == MOE_F32 ? 4 : t == MOE_BF16 || t == MOE_F16 ? 2 : 0; }

moe_status check_rule(const moe_route_rule* r, int T, int E, int k) {
    if (T < 0 || E <= 0 || E > kMaxE || k <= 0 || k > kMaxK || k > E) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!r) return MOE_ERR_INVALID_ARG;
    if (r->score != MOE_SCORE_SIGMOID && r->score != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID_ARG;
    if (r->group_score != MOE_GROUP_MAX && r->group_score != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARG;
    if (!isfinite(r->scale)) return MOE_ERR_INVALID_ARG;
    if (r->groups < 1 || r->groups > kMaxGroups || E % r->groups != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (r->top_groups < 1 || r->top_groups > r->groups) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (k > r->top_groups * (E / r->groups)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)T * k > (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// sizes whose padded products and tile counts stay far inside 64 and 32 bits
constexpr int64_t kMaxDim = (int64_t)1 << 28, kMaxArea = (int64_t)1 << 40;
bool dims_ok(int64_t a, int64_t b) { return a >= 0 && b >= 1 && a <= kMaxDim && b <= kMaxDim && a * b <= kMaxArea; }

moe_status check_operand(const moe_nvfp4_operand* o) {
    if (!o || !o->q || !o->s || !o->gs) return MOE_ERR_INVALID_ARG;
    if (!aligned(o->q, 16) || !aligned(o->s, 16) || !aligned(o->gs, 4)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

size_t pad(int64_t v, int64_t a) { return (size_t)((v + a - 1) / a * a); }

// Workspace of the dense products: control block, maxima of a two-form quantisation, the operand of x [M][K].
struct LinearLayout {
    size_t maxima, q, s, gs, total;
};
LinearLayout linear_layout(int64_t M, int64_t N, int64_t K) {
    LinearLayout L;
    const int64_t least = M < N ? (M < K ? M : K) : (N < K ? N : K);
    L.maxima = sizeof(Ctrl);
    L.q = align_up(L.maxima + 4 * (size_t)(M + N + K - least), 256);  // the largest sum of two of them
    L.s = align_up(L.q + moe_nvfp4_operand_codes(M, K), 256);
    L.gs = align_up(L.s + moe_nvfp4_operand_scales(M, K), 256);
    L.total = align_up(L.gs + 4 * (size_t)M, 256);
    return L;
}

moe_status check_workspace(void* ws, size_t ws_bytes, size_t need) {
    return ws == nullptr || !aligned(ws, 256) || ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

bool product_ok(int64_t M, int64_t N, int64_t K) { return dims_ok(M, K) && dims_ok(N, K) && dims_ok(M, N > 0 ? N : 1); }

moe_status check_product(int64_t M, int64_t N, int64_t K, const void* y, moe_dtype dtype, int64_t ldy) {
    if (!product_ok(M, N, K)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dtype_size(dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MOE_OK;
    if (ldy < N) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!y || !aligned(y, dtype_size(dtype))) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_route_logits(const uint16_t* x, const float* W_r, const float* b, int T, int d, int E, float* logits,
                            moe_stream_t stream) {
    MOE_TRY(check_shape(T, d, E, 1, 32, MOE_ACT_BF16));
    if (T == 0) return MOE_OK;
    if (!x || !W_r || !logits || !aligned(x, 16) || !aligned(W_r, 16) || !words(b, logits)) return MOE_ERR_INVALID_ARG;
    return launch([&] { return launch_route_logits(x, W_r, b, T, d, E, logits, (cudaStream_t)stream, false); });
}

moe_status moe_route_scores(const void* logits, moe_dtype dtype, int64_t ld, const float* bias, int T, int E, int k,
                            const moe_route_rule* rule, int32_t* ids, float* w, float* scores, int32_t* counts,
                            moe_stream_t stream) {
    MOE_TRY(check_rule(rule, T, E, k));
    if (dtype_size(dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (ld < E) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T > 0 && (!logits || !ids || !w || !aligned(logits, dtype_size(dtype)))) return MOE_ERR_INVALID_ARG;
    if (!words(bias, ids, w, scores, counts)) return MOE_ERR_INVALID_ARG;
    if (T == 0 && !counts) return MOE_OK;
    return launch([&] {
        cudaStream_t st = (cudaStream_t)stream;
        if (counts) {
            cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)E, st);
            if (e != cudaSuccess) return e;
        }
        RouteScoresArgs a = {logits, ld, bias, T, E, k, *rule, ids, w, scores, counts};
        return launch_route_scores(a, dtype, st);
    });
}

moe_status moe_route_scores_backward(const void* logits, moe_dtype dtype, int64_t ld, int T, int E, int k,
                                     const moe_route_rule* rule, const int32_t* ids, const float* dw, const float* dscores,
                                     void* dlogits, int64_t ldd, moe_stream_t stream) {
    MOE_TRY(check_rule(rule, T, E, k));
    if (dtype_size(dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (ld < E || ldd < E) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !ids || !dw || !dlogits || !aligned(logits, dtype_size(dtype)) || !aligned(dlogits, dtype_size(dtype)) ||
        !words(ids, dw, dscores))
        return MOE_ERR_INVALID_ARG;
    return launch([&] {
        RouteBackwardArgs a = {logits, ld, T, E, k, *rule, ids, dw, dscores, dlogits, ldd};
        return launch_route_scores_backward(a, dtype, (cudaStream_t)stream);
    });
}

moe_status moe_combine_backward(const uint16_t* dy, const uint16_t* y_perm, const int32_t* inv_pos, const float* w, int T,
                                int k, int d, float* dw, uint16_t* dy_perm, moe_stream_t stream) {
    if (T < 0 || k <= 0 || k > kMaxK || d <= 0 || d % 8 != 0 || (int64_t)T * k > (int64_t)1 << 30)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!dy || !inv_pos || !aligned(dy, 16) || (!dw && !dy_perm)) return MOE_ERR_INVALID_ARG;
    if (dw && (!y_perm || !aligned(y_perm, 16))) return MOE_ERR_INVALID_ARG;
    if (dy_perm && (!w || !aligned(dy_perm, 16))) return MOE_ERR_INVALID_ARG;
    if (!words(inv_pos, w, dw)) return MOE_ERR_INVALID_ARG;
    return launch([&] { return launch_combine_backward(dy, y_perm, inv_pos, w, T, k, d, dw, dy_perm, (cudaStream_t)stream); });
}

size_t moe_nvfp4_operand_codes(int64_t rows, int64_t K) { return dims_ok(rows, K) ? pad(rows, 128) * pad(K, 256) / 2 : 0; }
size_t moe_nvfp4_operand_scales(int64_t rows, int64_t K) { return dims_ok(rows, K) ? pad(rows, 128) * pad(K, 256) / 16 : 0; }

size_t moe_nvfp4_workspace_size(int64_t M, int64_t N, int64_t K) { return product_ok(M, N, K) ? linear_layout(M, N, K).total : 0; }

moe_status moe_nvfp4_quantize(const void* x, moe_dtype dtype, int64_t R, int64_t C, int64_t ld,
                              const moe_nvfp4_operand* rows, const moe_nvfp4_operand* cols, int scales_given, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
    if (!dims_ok(R, C) || ld < C) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dtype_size(dtype) == 0 || (!rows && !cols)) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    if (!x || !aligned(x, dtype_size(dtype))) return MOE_ERR_INVALID_ARG;
    for (const moe_nvfp4_operand* o : {rows, cols}) {
        if (!o) continue;
        MOE_TRY(check_operand(o));
        if (!scales_given && !o->gs_rows) return MOE_ERR_INVALID_ARG;
    }
    const bool scratch = cols && !scales_given;
    if (scratch) MOE_TRY(check_workspace(ws, ws_bytes, sizeof(Ctrl) + 4 * (size_t)((rows ? R : 0) + C)));
    return launch([&] {
        return launch_nvfp4_quantize(x, dtype, R, C, ld, rows, cols, scales_given != 0,
                                     scratch ? static_cast<char*>(ws) + sizeof(Ctrl) : nullptr, (cudaStream_t)stream);
    });
}

moe_status moe_nvfp4_operand_values(const moe_nvfp4_operand* op, int64_t rows, int64_t K, float* v, moe_stream_t stream) {
    if (!dims_ok(rows, K)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOE_OK;
    MOE_TRY(check_operand(op));
    if (!v || !aligned(v, 4)) return MOE_ERR_INVALID_ARG;
    return launch([&] { return launch_nvfp4_values(op, rows, K, v, (cudaStream_t)stream); });
}

moe_status moe_nvfp4_matmul(const moe_nvfp4_operand* A, const moe_nvfp4_operand* B, int64_t M, int64_t N, int64_t K, void* y,
                            moe_dtype dtype, int64_t ldy, void* ws, size_t ws_bytes, moe_stream_t stream) {
    MOE_TRY(check_product(M, N, K, y, dtype, ldy));
    if (M == 0 || N == 0) return MOE_OK;
    MOE_TRY(check_operand(A));
    MOE_TRY(check_operand(B));
    MOE_TRY(check_workspace(ws, ws_bytes, sizeof(Ctrl)));
    return launch([&] {
        return launch_nvfp4_matmul(A, B, M, N, K, y, dtype, ldy, &static_cast<Ctrl*>(ws)->status, (cudaStream_t)stream, false);
    });
}

moe_status moe_nvfp4_linear(const void* x, moe_dtype x_dtype, int64_t M, int64_t K, int64_t ldx, const moe_nvfp4_operand* W,
                            int64_t N, void* y, moe_dtype y_dtype, int64_t ldy, void* ws, size_t ws_bytes,
                            moe_stream_t stream) {
    MOE_TRY(check_product(M, N, K, y, y_dtype, ldy));
    if (dtype_size(x_dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (ldx < K) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return MOE_OK;
    if (!x || !aligned(x, dtype_size(x_dtype))) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_operand(W));
    const LinearLayout L = linear_layout(M, N, K);
    MOE_TRY(check_workspace(ws, ws_bytes, L.total));
    return launch([&] {
        char* base = static_cast<char*>(ws);
        const moe_nvfp4_operand A = {reinterpret_cast<uint8_t*>(base + L.q), reinterpret_cast<uint8_t*>(base + L.s),
                                     reinterpret_cast<float*>(base + L.gs), 1};
        cudaStream_t st = (cudaStream_t)stream;
        int* status = &static_cast<Ctrl*>(ws)->status;
        cudaError_t e = launch_nvfp4_quantize(x, x_dtype, M, K, ldx, &A, nullptr, false, nullptr, st);
        if (e != cudaSuccess) return e;
        return launch_nvfp4_matmul(&A, W, M, N, K, y, y_dtype, ldy, status, st, true);
    });
}

}  // extern "C"
