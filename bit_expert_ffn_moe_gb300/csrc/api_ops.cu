// api_ops.cu -- extern "C" entry points beside the layer (include/moe.h): routing rules and their gradient, the
// weighted sum's gradients, dense NVFP4 products, rows between tokens and experts, 8-bit products.  Argument checks and launches; nothing allocates device
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

bool expert_rows_ok(int T, int k, int d) {
    return T >= 0 && k >= 1 && k <= kMaxK && d >= 1 && (int64_t)T * k <= (int64_t)1 << 30 && (int64_t)T * k * d <= (int64_t)1 << 38;
}
bool experts_ok(int E) { return E >= 1 && E <= kMaxE; }
// A matrix of `dtype` with rows of n elements, ld apart.
bool matrix_ok(const void* p, moe_dtype dtype, int64_t n, int64_t ld) { return p && ld >= n && aligned(p, dtype_size(dtype)); }

constexpr int64_t kInt8MaxK = 131072;  // sums of K products of 127 x 127 stay below 2^31
bool int8_ok(int64_t rows, int64_t K) { return K <= kInt8MaxK && dims_ok(rows, K); }
// What a room has beyond the rows it is for, at most: so any room of accepted rows has bytes, and a workspace never lacks them.
constexpr int64_t kInt8Beside = 8 * (int64_t)kMaxE + 16 + 7;
bool int8_room_ok(int64_t room, int64_t K) { return room >= 0 && int8_ok(room > kInt8Beside ? room - kInt8Beside : 0, K); }
bool int8_product_ok(int64_t M, int64_t N, int64_t K) { return int8_ok(M, K) && int8_ok(N, K) && dims_ok(M, N > 0 ? N : 1); }

moe_status check_int8_weights(const moe_int8_weights* W) {
    return !W || !W->q || !W->s || !aligned(W->q, 16) || !aligned(W->s, 4) ? MOE_ERR_INVALID_ARG : MOE_OK;
}
moe_status check_int8_rows(const moe_int8_rows* r, int64_t M, int E) {
    if (!r || !r->q || !r->s || !aligned(r->q, 16) || !aligned(r->s, 4)) return MOE_ERR_INVALID_ARG;
    return r->room < moe_int8_rows_room(M, E) || r->room % 8 != 0 ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

// Workspaces of the 8-bit products: control block, shared tiles' partial sums, rows of x; and for a sparse layer the order, h and its
// rows, the experts' outputs.
struct Int8Layout {
    size_t partials, q, s, total;
};
Int8Layout int8_layout(int64_t M, int64_t K) {
    Int8Layout L;
    const int64_t room = moe_int8_rows_room(M, 0);
    L.partials = sizeof(Ctrl);
    L.q = align_up(L.partials + int8_partial_bytes(M), 256);
    L.s = align_up(L.q + moe_int8_rows_bytes(room, K), 256);
    L.total = align_up(L.s + 4 * (size_t)room, 256);
    return L;
}
struct Int8ExpertsLayout {
    int64_t room;
    size_t partials, offsets, inv, xq, xs, h, hq, hs, rows, total;
};
Int8ExpertsLayout int8_experts_layout(int T, int d, int E, int k, int I, moe_dtype dtype) {
    Int8ExpertsLayout L;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at = align_up(at + bytes, 256);
        return here;
    };
    const int64_t P = (int64_t)T * k;
    L.room = moe_int8_rows_room(P, E);
    take(sizeof(Ctrl));
    L.partials = take(int8_partial_bytes(P));
    L.offsets = take(4 * ((size_t)E + 1));
    L.inv = take(4 * (size_t)P);
    L.xq = take(moe_int8_rows_bytes(L.room, d));
    L.xs = take(4 * (size_t)L.room);
    L.h = take(dtype_size(dtype) * P * I);
    L.hq = take(moe_int8_rows_bytes(L.room, I));
    L.hs = take(4 * (size_t)L.room);
    L.rows = take(dtype_size(dtype) * P * d);
    L.total = at;
    return L;
}
bool int8_experts_ok(int T, int d, int E, int k, int I) {
    return experts_ok(E) && d >= 1 && I >= 1 && expert_rows_ok(T, k, d) && expert_rows_ok(T, k, I) && I <= (1 << 27) &&
           int8_product_ok((int64_t)T * k, 2 * (int64_t)I, d) && int8_product_ok((int64_t)T * k, d, I);
}

moe_status check_int8_pack(const void* w, int E, int64_t rows, int64_t K, int64_t ld, int64_t first, int64_t step, int64_t N,
                           const moe_int8_weights* W) {
    if (!int8_ok(N, K) || rows < 0 || rows > N || E < 0 || E > kMaxE || ld < K || E * rows > (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (first < 0 || step < 1 || step > N || (rows > 0 && first + step * (rows - 1) >= N)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (E == 0 || rows == 0) return MOE_OK;
    return w ? check_int8_weights(W) : MOE_ERR_INVALID_ARG;
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

moe_status moe_expert_order(const int32_t* ids, int T, int k, int E, int32_t* offsets, int32_t* inv, moe_stream_t stream) {
    if (!expert_rows_ok(T, k, 1) || !experts_ok(E)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!offsets || (T > 0 && (!ids || !inv)) || !words(ids, offsets, inv)) return MOE_ERR_INVALID_ARG;
    return launch([&] { return launch_expert_order(ids, T * k, E, offsets, inv, (cudaStream_t)stream); });
}

moe_status moe_tokens_to_experts(const void* x, moe_dtype dtype, int64_t ldx, const int32_t* inv, const float* w, int T, int k, int d,
                                 void* rows, int64_t ldr, moe_stream_t stream) {
    if (!expert_rows_ok(T, k, d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dtype_size(dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (ldx < d || ldr < d) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!matrix_ok(x, dtype, d, ldx) || !matrix_ok(rows, dtype, d, ldr) || !inv || !words(inv, w)) return MOE_ERR_INVALID_ARG;
    return launch([&] {
        return launch_expert_rows(true, dtype, x, ldx, nullptr, 0, rows, ldr, inv, w, nullptr, T, k, d, (cudaStream_t)stream);
    });
}

moe_status moe_tokens_to_experts_backward(const void* drows, moe_dtype dtype, int64_t ldr, const void* x, int64_t ldx,
                                          const int32_t* inv, const float* w, int T, int k, int d, void* dx, int64_t ldd, float* dw,
                                          moe_stream_t stream) {
    if (!expert_rows_ok(T, k, d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dtype_size(dtype) == 0 || (!dx && !dw)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (ldr < d || (dx && ldd < d) || (dw && ldx < d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!matrix_ok(drows, dtype, d, ldr) || (dx && !matrix_ok(dx, dtype, d, ldd)) || (dw && !matrix_ok(x, dtype, d, ldx)) || !inv ||
        !words(inv, w, dw))
        return MOE_ERR_INVALID_ARG;
    return launch([&] {
        return launch_expert_rows(false, dtype, dw ? x : nullptr, ldx, drows, ldr, dx, ldd, inv, w, dw, T, k, d, (cudaStream_t)stream);
    });
}

moe_status moe_experts_to_tokens(const void* rows, moe_dtype dtype, int64_t ldr, const int32_t* inv, const float* w, int T, int k,
                                 int d, void* y, int64_t ldy, moe_stream_t stream) {
    if (!expert_rows_ok(T, k, d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dtype_size(dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (ldr < d || ldy < d) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!matrix_ok(rows, dtype, d, ldr) || !matrix_ok(y, dtype, d, ldy) || !inv || !words(inv, w)) return MOE_ERR_INVALID_ARG;
    return launch([&] {
        return launch_expert_rows(false, dtype, nullptr, 0, rows, ldr, y, ldy, inv, w, nullptr, T, k, d, (cudaStream_t)stream);
    });
}

moe_status moe_experts_to_tokens_backward(const void* dy, moe_dtype dtype, int64_t ldy, const void* rows, int64_t ldr,
                                          const int32_t* inv, const float* w, int T, int k, int d, void* drows, int64_t ldg, float* dw,
                                          moe_stream_t stream) {
    if (!expert_rows_ok(T, k, d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dtype_size(dtype) == 0 || (!drows && !dw)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (ldy < d || (drows && ldg < d) || (dw && ldr < d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!matrix_ok(dy, dtype, d, ldy) || (drows && !matrix_ok(drows, dtype, d, ldg)) || (dw && !matrix_ok(rows, dtype, d, ldr)) || !inv ||
        !words(inv, w, dw))
        return MOE_ERR_INVALID_ARG;
    return launch([&] {
        return launch_expert_rows(true, dtype, dy, ldy, dw ? rows : nullptr, ldr, drows, ldg, inv, w, dw, T, k, d, (cudaStream_t)stream);
    });
}

size_t moe_int8_weights_bytes(int64_t N, int64_t K) { return int8_ok(N, K) ? (size_t)int8_tiles(N, K) * kInt8Tile : 0; }
int64_t moe_int8_rows_room(int64_t M, int E) {
    return M < 0 || M > kMaxDim || E < 0 || E > kMaxE ? 0 : (M + 7) / 8 * 8 + 8 * (int64_t)E + 16;
}
size_t moe_int8_rows_bytes(int64_t room, int64_t K) { return int8_room_ok(room, K) ? (size_t)room * pad(K, 64) * 2 : 0; }

moe_status moe_int8_weights_layout(const int8_t* w, const float* s_in, int E, int64_t rows, int64_t K, int64_t ld, int64_t first,
                                   int64_t step, int64_t N, const moe_int8_weights* W, moe_stream_t stream) {
    MOE_TRY(check_int8_pack(w, E, rows, K, ld, first, step, N, W));
    if (E == 0 || rows == 0) return MOE_OK;
    if (!s_in || !words(s_in)) return MOE_ERR_INVALID_ARG;
    return launch([&] {
        return launch_int8_pack({w, s_in, E, rows, K, ld, (int)first, (int)step, N, const_cast<uint8_t*>(W->q), const_cast<float*>(W->s)}, -1,
                                (cudaStream_t)stream);
    });
}

moe_status moe_int8_weights_quantize(const void* w, moe_dtype dtype, int E, int64_t rows, int64_t K, int64_t ld, int64_t first,
                                     int64_t step, int64_t N, const moe_int8_weights* W, moe_stream_t stream) {
    if (dtype_size(dtype) == 0) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_int8_pack(w, E, rows, K, ld, first, step, N, W));
    if (E == 0 || rows == 0) return MOE_OK;
    if (!aligned(w, dtype_size(dtype))) return MOE_ERR_INVALID_ARG;
    return launch([&] {
        return launch_int8_pack({w, nullptr, E, rows, K, ld, (int)first, (int)step, N, const_cast<uint8_t*>(W->q), const_cast<float*>(W->s)},
                                dtype, (cudaStream_t)stream);
    });
}

moe_status moe_int8_quantize(const void* x, moe_dtype dtype, int64_t T, int64_t K, int64_t ldx, const int32_t* inv, int k,
                             const int32_t* offsets, int E, const moe_int8_rows* rows, moe_stream_t stream) {
    if (dtype_size(dtype) == 0 || (inv && !offsets) || (offsets ? !experts_ok(E) : E != 0)) return MOE_ERR_INVALID_ARG;
    if (inv && (k < 1 || k > kMaxK)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T < 0 || T > kMaxDim) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t M = inv ? T * k : T;
    if (M > kMaxDim || !int8_ok(M, K)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (ldx < K) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!matrix_ok(x, dtype, K, ldx) || !words(inv, offsets)) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_int8_rows(rows, M, E));
    return launch([&] {
        return launch_int8_rows({x, ldx, T, K, inv, k, offsets, E, rows->room, rows->q, rows->s}, dtype, (cudaStream_t)stream);
    });
}

size_t moe_int8_workspace_size(int64_t M, int64_t N, int64_t K) { return int8_product_ok(M, N, K) ? int8_layout(M, K).total : 0; }

moe_status moe_int8_matmul(const moe_int8_rows* rows, const int32_t* offsets, int E, int64_t M, const moe_int8_weights* W, int64_t N,
                           int64_t K, int gated, void* y, moe_dtype dtype, int64_t ldy, void* ws, size_t ws_bytes,
                           moe_stream_t stream) {
    if (!int8_product_ok(M, N, K) || (gated && N % 2 != 0)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (offsets ? !experts_ok(E) || !words(offsets) : E != 0) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_product(M, gated ? N / 2 : N, K, y, dtype, ldy));
    if (M == 0 || N == 0) return MOE_OK;
    MOE_TRY(check_int8_weights(W));
    MOE_TRY(check_int8_rows(rows, M, E));
    const Int8Layout L = int8_layout(M, K);
    MOE_TRY(check_workspace(ws, ws_bytes, L.q));
    return launch([&] {
        return launch_int8_product({W->q, W->s, rows->q, rows->s, rows->room, offsets, offsets ? E : 1, M, N, K, y, ldy, static_cast<Ctrl*>(ws),
                                    reinterpret_cast<float*>(static_cast<char*>(ws) + L.partials), 0},
                                   dtype, gated != 0, (cudaStream_t)stream);
    });
}

moe_status moe_int8_linear(const void* x, moe_dtype x_dtype, int64_t M, int64_t K, int64_t ldx, const moe_int8_weights* W, int64_t N,
                           int gated, void* y, moe_dtype y_dtype, int64_t ldy, void* ws, size_t ws_bytes, moe_stream_t stream) {
    if (!int8_product_ok(M, N, K) || (gated && N % 2 != 0)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dtype_size(x_dtype) == 0) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_product(M, gated ? N / 2 : N, K, y, y_dtype, ldy));
    if (M == 0 || N == 0) return MOE_OK;
    if (ldx < K) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!matrix_ok(x, x_dtype, K, ldx)) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_int8_weights(W));
    const Int8Layout L = int8_layout(M, K);
    MOE_TRY(check_workspace(ws, ws_bytes, L.total));
    return launch([&] {
        char* base = static_cast<char*>(ws);
        cudaStream_t st = (cudaStream_t)stream;
        const int64_t room = moe_int8_rows_room(M, 0);
        uint16_t* q = reinterpret_cast<uint16_t*>(base + L.q);
        float* s = reinterpret_cast<float*>(base + L.s);
        return launch_int8_linear(x, x_dtype, ldx, q, s,
                                  {W->q, W->s, nullptr, nullptr, room, nullptr, 1, M, N, K, y, ldy, static_cast<Ctrl*>(ws),
                                   reinterpret_cast<float*>(base + L.partials), 0},
                                  y_dtype, gated != 0, st);
    });
}

size_t moe_int8_experts_workspace_size(int T, int d, int E, int k, int I, moe_dtype dtype) {
    return int8_experts_ok(T, d, E, k, I) && dtype_size(dtype) != 0 ? int8_experts_layout(T, d, E, k, I, dtype).total : 0;
}

moe_status moe_int8_experts(const void* x, moe_dtype dtype, int64_t ldx, const int32_t* ids, const float* w, int T, int d, int E, int k,
                            int I, const moe_int8_weights* up, const moe_int8_weights* down, void* y, int64_t ldy, void* ws,
                            size_t ws_bytes, moe_stream_t stream) {
    if (!int8_experts_ok(T, d, E, k, I)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dtype_size(dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (ldx < d || ldy < d) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!matrix_ok(x, dtype, d, ldx) || !matrix_ok(y, dtype, d, ldy) || !ids || !w || !words(ids, w)) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_int8_weights(up));
    MOE_TRY(check_int8_weights(down));
    const Int8ExpertsLayout L = int8_experts_layout(T, d, E, k, I, dtype);
    MOE_TRY(check_workspace(ws, ws_bytes, L.total));
    return launch([&] {
        char* base = static_cast<char*>(ws);
        cudaStream_t st = (cudaStream_t)stream;
        const int64_t P = (int64_t)T * k;
        int32_t* offsets = reinterpret_cast<int32_t*>(base + L.offsets);
        int32_t* inv = reinterpret_cast<int32_t*>(base + L.inv);
        uint16_t *xq = reinterpret_cast<uint16_t*>(base + L.xq), *hq = reinterpret_cast<uint16_t*>(base + L.hq);
        float *xs = reinterpret_cast<float*>(base + L.xs), *hs = reinterpret_cast<float*>(base + L.hs);
        Ctrl* ctrl = static_cast<Ctrl*>(ws);
        float* partials = reinterpret_cast<float*>(base + L.partials);
        cudaError_t e = launch_expert_order(ids, (int)P, E, offsets, inv, st);
        if (e == cudaSuccess)
            e = launch_int8_by_expert(x, ldx, T, inv, k, xq, xs, {up->q, up->s, nullptr, nullptr, L.room, offsets, E, P, 2 * (int64_t)I, d,
                                                                  base + L.h, I, ctrl, partials, 0},
                                      dtype, true, st);
        if (e == cudaSuccess)  // (the kernel in front has waited for the order)
            e = launch_int8_by_expert(base + L.h, I, P, nullptr, 1, hq, hs, {down->q, down->s, nullptr, nullptr, L.room, offsets, E, P, d, I,
                                                                             base + L.rows, d, ctrl, partials, 1},
                                      dtype, false, st);
        if (e == cudaSuccess)
            e = launch_expert_rows(false, dtype, nullptr, 0, base + L.rows, d, y, ldy, inv, w, nullptr, T, k, d, st);
        return e;
    });
}

}  // extern "C"
