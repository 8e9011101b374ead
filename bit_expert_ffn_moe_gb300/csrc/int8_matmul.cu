// int8_matmul.cu -- products of 8-bit rows and 8-bit weights, of all rows with one matrix or of each expert's rows with its own:
//   y[m][n] = (sum_k qx[m][k] qw[n][k]) sx[m] sw[n]
// or gated, for rows 2 i and 2 i + 1 of the weights (gate and up of channel i):  y[m][i] = silu(gate) up.
// The sum of whole numbers is exact up to 2^24 and rounded to fp32 beyond; the two products with the scales are in fp32, in this
// order, and the result is rounded once to y's type.
//
//   mma     (int8_mma.cu) the tensor cores, on fp16 that holds the whole numbers
//   dot     few rows: dot products of four bytes (dp4a), the weights read once.  The rows of all active experts' matrices are
//           dealt out evenly to the CTAs, so that no partial sums have to be exchanged; a warp takes every 16th step of 64 values
//           of 32 weight rows.
#include "int8_common.cuh"

namespace moe {
namespace {

constexpr int kDotThreads = 512, kDotWarps = kDotThreads / 32;
constexpr int kDotRows = 32;     // weight rows at a time
constexpr int kDotTokens = 4;    // activation rows at a time
constexpr int kDotK = 16384;     // values of them in shared memory at a time

// Four fp16 whole numbers as four bytes.
__device__ __forceinline__ uint32_t bytes_of(uint2 h) {
    const __half2 a = *reinterpret_cast<const __half2*>(&h.x), b = *reinterpret_cast<const __half2*>(&h.y);
    return (uint32_t)(__half2int_rn(__low2half(a)) & 255) | ((uint32_t)(__half2int_rn(__high2half(a)) & 255) << 8) |
           ((uint32_t)(__half2int_rn(__low2half(b)) & 255) << 16) | ((uint32_t)(__half2int_rn(__high2half(b)) & 255) << 24);
}

// Steps kt0 .. kt1 of 64 values: the warp's share of up to 32 weight rows times TM activation rows.  Lane (i, j) = (lane % 8, lane / 8)
// takes the 16 bytes j of rows i, i + 8, i + 16, i + 24 (row[g] null: none).
template <int TM>
__device__ __forceinline__ void dot_steps(const uint8_t* const (&row)[4], const uint8_t* x, int kt0, int kt1, int (&acc)[4][kDotTokens]) {
    const int warp = threadIdx.x >> 5, j = (threadIdx.x & 31) >> 3;
    for (int kt = kt0 + warp; kt < kt1; kt += 4 * kDotWarps) {
        uint4 w[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int at = kt + u * kDotWarps;
                w[u][g] = row[g] && at < kt1 ? ldg_stream(row[g] + (int64_t)at * kInt8Tile) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int at = kt + u * kDotWarps;
            if (at >= kt1) break;
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                const uint4 v = *reinterpret_cast<const uint4*>(x + t * kDotK + (at - kt0) * 64 + j * 16);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    acc[g][t] = __dp4a((int)w[u][g].x, (int)v.x, acc[g][t]);
                    acc[g][t] = __dp4a((int)w[u][g].y, (int)v.y, acc[g][t]);
                    acc[g][t] = __dp4a((int)w[u][g].z, (int)v.z, acc[g][t]);
                    acc[g][t] = __dp4a((int)w[u][g].w, (int)v.w, acc[g][t]);
                }
            }
        }
    }
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(kDotThreads, 1) int8_dot_kernel(const Int8ProductArgs a) {
    extern __shared__ __align__(16) uint8_t x[];  // [kDotTokens][kDotK]
    __shared__ int red[kDotWarps][kDotRows][kDotTokens];
    __shared__ int active[kMaxE + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {  // the experts that have rows
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const bool has = e < a.E && (a.offsets ? __ldg(a.offsets + e + 1) > __ldg(a.offsets + e) : a.M > 0);
            const unsigned b = __ballot_sync(0xffffffffu, has);
            if (has) active[n + __popc(b & ((1u << lane) - 1u))] = e;
            n += __popc(b);
        }
        if (lane == 0) active[kMaxE] = n;
    }
    __syncthreads();
    const int KT = (int)((a.K + 63) / 64);
    const int64_t NP = (a.N + 1) / 2, pairs = NP * active[kMaxE];  // weight rows are dealt out in twos
    const int64_t end = pairs * (blockIdx.x + 1) / gridDim.x;
    for (int64_t at = pairs * blockIdx.x / gridDim.x; at < end;) {
        const int e = active[at / NP];
        const int64_t n0 = 2 * (at % NP), n1 = min(a.N, n0 + 2 * (end - at));
        at += NP - at % NP;
        const int64_t first = a.offsets ? a.offsets[e] : 0, count = a.offsets ? a.offsets[e + 1] - first : a.M;
        const int64_t row0 = a.offsets ? int8_first_row(first, e) : 0;
        const uint8_t* we = a.w + (int64_t)e * int8_tiles(a.N, a.K) * kInt8Tile;
        for (int64_t t0 = 0; t0 < count; t0 += kDotTokens) {
            const int tokens = (int)min((int64_t)kDotTokens, count - t0);
            int have = -1;  // the step from which on shared memory holds these rows
            for (int64_t n = n0; n < n1; n += kDotRows) {
                const uint8_t* row[4];
                int acc[4][kDotTokens] = {};
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int64_t r = n + (lane & 7) + 8 * g;
                    row[g] = r < n1 ? we + (r / 128) * KT * kInt8Tile + (r % 128) * 16 + (lane >> 3) * 2048 : nullptr;
                }
                for (int k0 = 0; k0 < KT; k0 += kDotK / 64) {
                    const int k1 = min(KT, k0 + kDotK / 64);
                    if (have != k0) {
                        __syncthreads();
                        for (int i = threadIdx.x; i < tokens * (k1 - k0) * 8; i += kDotThreads) {
                            const int t = i / ((k1 - k0) * 8), c = i % ((k1 - k0) * 8);
                            const int64_t r = row0 + t0 + t;
                            const uint4 h = *reinterpret_cast<const uint4*>(a.x + ((int64_t)(k0 + c / 8) * a.room + r) * 64 +
                                                                            ((c % 8) ^ (int)(r % 8)) * 8);
                            *reinterpret_cast<uint2*>(x + t * kDotK + c * 8) =
                                make_uint2(bytes_of(make_uint2(h.x, h.y)), bytes_of(make_uint2(h.z, h.w)));
                        }
                        __syncthreads();
                        have = k0;
                    }
                    if (tokens == 1) dot_steps<1>(row, x, k0, k1, acc);
                    else if (tokens == 2) dot_steps<2>(row, x, k0, k1, acc);
                    else dot_steps<4>(row, x, k0, k1, acc);
                }
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int t = 0; t < kDotTokens; ++t) {
                        int v = acc[g][t];
                        v += __shfl_xor_sync(0xffffffffu, v, 8);
                        v += __shfl_xor_sync(0xffffffffu, v, 16);
                        if (lane < 8) red[warp][lane + 8 * g][t] = v;
                    }
                __syncthreads();
                const int t = threadIdx.x / kDotRows, r = threadIdx.x % kDotRows;
                if (t < tokens && n + r < n1 && (!GATED || r % 2 == 0)) {
                    int s0 = 0, s1 = 0;
                    for (int w = 0; w < kDotWarps; ++w) {
                        s0 += red[w][r][t];
                        if (GATED) s1 += red[w][r + 1][t];
                    }
                    const float sx = a.sx[row0 + t0 + t];
                    const float* sw = a.sw + (int64_t)e * a.N + n + r;
                    const float v = (float)s0 * sx * sw[0];
                    T* y = static_cast<T*>(a.y) + (first + t0 + t) * a.ldy;
                    if (GATED) y[(n + r) / 2] = int8_result<T>(int8_gated(v, (float)s1 * sx * sw[1]));
                    else y[n + r] = int8_result<T>(v);
                }
                __syncthreads();
            }
        }
    }
}

template <bool GATED>
const void* dot_kernel(moe_dtype dtype) {
    return dtype == MOE_F32    ? (const void*)int8_dot_kernel<float, GATED>
           : dtype == MOE_BF16 ? (const void*)int8_dot_kernel<__nv_bfloat16, GATED>
                               : (const void*)int8_dot_kernel<__half, GATED>;
}

}  // namespace

cudaError_t launch_int8_dot(const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st) {
    void* args[] = {const_cast<Int8ProductArgs*>(&a)};
    return launch_kernel(gated ? dot_kernel<true>(dtype) : dot_kernel<false>(dtype), dim3(sm_count()), dim3(kDotThreads),
                         kDotTokens * kDotK, st, true, args);
}

cudaError_t launch_int8_product(const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st) {
    if (a.M == 0 || a.N == 0) return cudaSuccess;
    // Us, dot / one CTA a tile / pairs: 1 x 4096 x 8192 9.6 / 17 / 18, 4 x 4096 x 8192 12.5 / 17 / 18, 16: 36 / 17 / 18; 128: 29 / 29, 256: 34 / 31,
    // 4096: 220 / 161; by expert, 128 of 4096 x 8192, a mean of 0.25 rows: 157 / 153 / 153, 4: 593 / 592, 16: 704 / 647, 64: 1041 / 805.
    if (a.M <= 4) return launch_int8_dot(a, dtype, gated, st);
    return launch_int8_mma(a, dtype, gated, a.offsets ? a.M / a.E >= 16 : a.M > 128, st);
}

}  // namespace moe
