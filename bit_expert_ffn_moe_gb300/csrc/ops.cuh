// ops.cuh -- launch entry points of the kernels beside the layer: routing rules and their gradient,
// the weighted sum's gradients, NVFP4 operands and their dense product (called by api_ops.cu).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxGroups = 32;  // expert groups of a routing rule: one lane each

struct RouteScoresArgs {
    const void* logits;  // [T][ld] of dtype
    int64_t ld;
    const float* bias;  // [E] or null
    int T, E, k;
    moe_route_rule rule;
    int32_t* ids;     // [T][k]
    float* w;         // [T][k]
    float* scores;    // [T][E] or null
    int32_t* counts;  // [E] or null (zeroed before the launch)
};
cudaError_t launch_route_scores(const RouteScoresArgs& a, moe_dtype dtype, cudaStream_t st);

struct RouteBackwardArgs {
    const void* logits;  // [T][ld] of dtype
    int64_t ld;
    int T, E, k;
    moe_route_rule rule;
    const int32_t* ids;    // [T][k]
    const float* dw;       // [T][k]
    const float* dscores;  // [T][E] or null
    void* dlogits;         // [T][ldd] of dtype
    int64_t ldd;
};
cudaError_t launch_route_scores_backward(const RouteBackwardArgs& a, moe_dtype dtype, cudaStream_t st);

cudaError_t launch_combine_backward(const uint16_t* dy, const uint16_t* y_perm, const int32_t* inv_pos, const float* w,
                                    int T, int k, int d, float* dw, uint16_t* dy_perm, cudaStream_t st);

// NVFP4 operands (nvfp4_operand.cu): of x [R][C] row by row (rows), column by column (cols), or both.  given: the
// operands' row scales are read, else computed.  maxima: R + C words, for cols with computed scales.
cudaError_t launch_nvfp4_quantize(const void* x, moe_dtype dtype, int64_t R, int64_t C, int64_t ld,
                                  const moe_nvfp4_operand* rows, const moe_nvfp4_operand* cols, bool given, void* maxima,
                                  cudaStream_t st);
cudaError_t launch_nvfp4_values(const moe_nvfp4_operand* op, int64_t R, int64_t K, float* v, cudaStream_t st);
// y [M][ldy] = A B^T (nvfp4_matmul.cu).  weights_ready: B does not come from the launch before, so its
// copies may start while that one runs.
cudaError_t launch_nvfp4_matmul(const moe_nvfp4_operand* A, const moe_nvfp4_operand* B, int64_t M, int64_t N, int64_t K, void* y,
                                moe_dtype dtype, int64_t ldy, int* status, cudaStream_t st, bool weights_ready);
}  // namespace moe
