// int8_matmul.cu -- products of 8-bit rows and 8-bit weights, of all rows with one matrix or of each expert's rows with its own:
//   y[m][n] = (sum_k qx[m][k] qw[n][k]) sx[m] sw[n]
// or gated, for rows 2 i and 2 i + 1 of the weights (gate and up of channel i):  y[m][i] = silu(gate) up.
// The sum of whole numbers is exact where it stays within 2^24 on its way (K <= 1032 always does).  Beyond, mma and few round their fp32
// accumulators as they add, 16 terms at a time: an adder that keeps at least 24 bits of the largest addend is off by less than 18 steps of
// 2^-23 of it, K / 16 times; so by less than K 2^-22 of the largest sum on the way.  (Accumulators taken out every 1024 values and added as
// whole numbers would be exact, but have no room beside the next tile's in tensor memory.)  dot adds whole numbers and rounds once.  The
// two products with the scales are in fp32, in this order, and the result is rounded once to y's type.
//
//   mma     (int8_mma.cu) the tensor cores, on fp16 that holds the whole numbers
//   few     (int8_few.cu) the same for one matrix and so few rows that there are no more tiles than SMs
//   dot     (int8_dot.cu) few rows: dot products of four bytes
#include "int8_common.cuh"

namespace moe {

constexpr int kDotRows = 4, kDotExpertRows = 32;

namespace {
// Few rows, and not so many to an expert that their dot products take longer than the weights' way.
bool few_by_expert(const Int8ProductArgs& a) { return a.M <= kDotExpertRows && a.M <= 8 * (int64_t)a.E; }
}  // namespace

cudaError_t launch_int8_product(const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st) {
    if (a.M == 0 || a.N == 0) return cudaSuccess;
    // us for 4096 x 8192 weights, dot / few / mma with one CTA a tile / with pairs: 1 row 10.2 / 12.0 / 17.4 / 18.6, 2: 10.9 / 12.0, 4: 12.5 / 12.0,
    // 16: 36 / 11.7 / 17.2 / 18.6, 128: - / 14.8 / 28.8 / 29.6, 512: - / 34.4 / 44.5 / 40.9, 4096: - / - / 220 / 160.  By expert, 128 of 4096 x 8192: 32 rows 147 / - / 155,
    // 64: 264 / - / 246; 2 of 2048 x 4096: 4 rows each 11.0 / - / 16.3, 15: 27.0 / - / 16.1; one CTA
    // a tile / pairs, 128 experts and a mean of 4 rows 593 / 592, 16: 704 / 647, 64: 1041 / 805.
    if (a.offsets ? few_by_expert(a) : a.M <= (int8_few_fits(a) ? 2 : kDotRows)) return launch_int8_dot(a, dtype, gated, nullptr, MOE_F32, 0, nullptr, 1, st);
    if (int8_few_fits(a)) return launch_int8_few(a, dtype, gated, st);
    return launch_int8_mma(a, dtype, gated, a.offsets ? a.M / a.E >= 16 : a.M > 128, st);
}

cudaError_t launch_int8_linear(const void* x, moe_dtype x_dtype, int64_t ldx, uint16_t* q, float* s, const Int8ProductArgs& a, moe_dtype dtype,
                               bool gated, cudaStream_t st) {
    if (a.M == 0 || a.N == 0) return cudaSuccess;
    // Every CTA quantises all of x for itself while its first weights arrive, which pays as long as x is short.  us of a call, x quantised by
    // the dot products / by the rows' kernel in front: 4096 x 8192 weights, 3 rows 14.4 / 13.5, 4: 14.8 / 13.5; x 5504, 3 rows 11.6 / 11.4, 4:
    // 11.9 / 11.4; 16384 x 8192, 3 rows 32.0 / 27.5; 4096 x 16384, 2 rows 19.7 / 21.1, 4: 24.0 / 19.1.  (2 rows of more than 8192 values lose by
    // it.  The dot products' room is for 4 rows of 16384.)
    if (a.M <= kDotRows && a.M * a.K <= kInt8DotK) return launch_int8_dot(a, dtype, gated, x, x_dtype, ldx, nullptr, 1, st);
    const cudaError_t e = launch_int8_rows({x, ldx, a.M, a.K, nullptr, 1, nullptr, 0, a.room, q, s}, x_dtype, st);
    if (e != cudaSuccess) return e;
    Int8ProductArgs p = a;
    p.x = q, p.sx = s;
    p.early = 1;  // (the rows' kernel has waited for what was in front of it)
    return launch_int8_product(p, dtype, gated, st);
}

cudaError_t launch_int8_by_expert(const void* x, int64_t ldx, int64_t T, const int32_t* inv, int k, uint16_t* q, float* s,
                                  const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st) {
    // Without kernels of the rows' own the layer of a token with 8 of 128 experts of 8192 x 2048 takes 79.1 us instead of 83.4.
    if (few_by_expert(a) && a.K <= kInt8DotK) return launch_int8_dot(a, dtype, gated, x, dtype, ldx, inv, k, st);
    const cudaError_t e = launch_int8_rows({x, ldx, T, a.K, inv, k, a.offsets, a.E, a.room, q, s}, dtype, st);
    if (e != cudaSuccess) return e;
    Int8ProductArgs p = a;
    p.x = q, p.sx = s;
    p.early = 1;  // (the rows' kernel has waited for what was in front of it)
    return launch_int8_product(p, dtype, gated, st);
}

}  // namespace moe
