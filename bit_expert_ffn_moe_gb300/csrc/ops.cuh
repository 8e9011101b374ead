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

// Pairs by expert (expert_order.cu), and rows between tokens and experts (expert_rows.cu): a the tokens' rows [T][lda], read
// (spread, dw), b rows [T k][ldb], read (gather, dw).
cudaError_t launch_expert_order(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* inv, cudaStream_t st);
cudaError_t launch_expert_rows(bool spread, moe_dtype dtype, const void* a, int64_t lda, const void* b, int64_t ldb, void* out,
                               int64_t ldo, const int32_t* inv, const float* w, float* dw, int T, int k, int d, cudaStream_t st);

// 8-bit operands (int8_operand.cu).
// Weights: tiles of 128 rows x 64 values, in a tile the 16-byte pieces j = 0 .. 3 of all rows next to each other.
constexpr int kInt8Tile = 128 * 64;
__host__ __device__ inline int64_t int8_tiles(int64_t N, int64_t K) { return ((N + 127) / 128) * ((K + 63) / 64); }
// Activations: fp16 numbers, [K / 64][rows][64], the 16-byte piece j of row r at place j ^ (r % 8) of its 128 bytes.  The rows of expert e
// start at a multiple of 8 that depends on its offset alone, behind those of the experts before: its offset rounded up, and 8 e.
__host__ __device__ inline int64_t int8_first_row(int64_t offset, int e) { return (offset + 7) / 8 * 8 + 8 * (int64_t)e; }

struct Int8PackArgs {
    const void* w;  // [E][rows][ld] of dtype, or int8 with its scales s_in [E][rows]
    const float* s_in;
    int E;
    int64_t rows, K, ld;
    int first, step;  // row i goes to row first + step i of N
    int64_t N;
    uint8_t* q;
    float* s;
};
cudaError_t launch_int8_pack(const Int8PackArgs& a, int dtype, cudaStream_t st);  // dtype < 0: int8
struct Int8RowsArgs {
    const void* x;  // [T][ld] of dtype
    int64_t ld;
    int64_t T, K;
    const int32_t* inv;  // [T][k]: the rows of a token in expert order; null: row t is row t
    int k;
    const int32_t* offsets;  // [E + 1]; null: one group
    int E;
    int64_t room;  // rows of the operand
    uint16_t* q;
    float* s;
};
cudaError_t launch_int8_rows(const Int8RowsArgs& a, moe_dtype dtype, cudaStream_t st);

// Products of 8-bit rows and weights (int8_matmul.cu), of all rows with one matrix (offsets null) or by expert.
struct Int8ProductArgs {
    const uint8_t* w;  // E matrices of int8_tiles(N, K) tiles
    const float* sw;   // [E][N]
    const uint16_t* x;
    const float* sx;
    int64_t room;
    const int32_t* offsets;
    int E;
    int64_t M;  // rows, or rows at most
    int64_t N, K;
    void* y;  // [M][ldy], N values a row, gated: N / 2
    int64_t ldy;
    Ctrl* ctrl;
    float* partials;  // int8_partial_bytes(M)
    int early;        // w, sw and offsets were there before the kernel in front started its dependents
};
// Partial sums of the tiles that CTAs share: two tiles of 128 weight rows a CTA, by as many activation rows as a tile has at most.
constexpr int kInt8Ctas = 160;  // CTAs at most
inline size_t int8_partial_bytes(int64_t M) { return (size_t)kInt8Ctas * 2 * 128 * 4 * (size_t)(M > 192 ? 192 : (M + 15) / 16 * 16); }
cudaError_t launch_int8_product(const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st);
// The same of rows x [a.M][ldx], quantised into q and s (a.room rows) where the product does not do it itself; a.early: whether w and
// sw were there before the kernel in front started its dependents.
cudaError_t launch_int8_linear(const void* x, moe_dtype x_dtype, int64_t ldx, uint16_t* q, float* s, const Int8ProductArgs& a, moe_dtype dtype,
                               bool gated, cudaStream_t st);
// The same by expert, of T rows x of the results' type: tokens that go to the rows inv [T][k] in expert order, or (inv null) rows in that
// order.  a.early as above, and for a.offsets.
cudaError_t launch_int8_by_expert(const void* x, int64_t ldx, int64_t T, const int32_t* inv, int k, uint16_t* q, float* s,
                                  const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st);
}  // namespace moe
