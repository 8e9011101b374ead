// nvfp4_operand.cu -- NVFP4 operands of the dense product: E2M1 codes, one E4M3 scale per 16 elements along
// the contraction and one fp32 scale per operand row, written straight in the tensor-core layout, from a
// matrix x [R][C] of fp32, bf16 or fp16 (row stride ld), its transpose, or both.
//
// The rule is the weight packer's, row by row: g = max|row| / 2688 (1 when 0); per block t = (max|block| / g) / 6,
// scale = nearest E4M3 (ties to even, saturating), D = scale * g, code = nearest E2M1 to v / D; every step
// in fp32, rounded to nearest even.  A row's own scale keeps a token's operand independent of the other
// tokens of its batch.
//
// v / D costs three fp32 operations: q0 = v y, q = q0 + (v - q0 D) y with y = 1 / D rounded (Markstein's
// correction, IBM J. Res. Dev. 34, 1990).  Over all 2^23 mantissas of D and all v within six ulps of the seven
// values where the code changes, q decides as the rounded quotient does (checked exhaustively on a CPU;
// without the correction 4% of those decisions differ), and farther away one ulp cannot change a
// code.  D outside 2^-60 .. 2^60 takes the division.
//
// Row form: the threads of a row read it once (K <= 8192: 32 elements each in registers), reduce its maximum and
// encode.  Both forms at once: two passes over x, the first for the row and column maxima (integer
// maxima of the bits: the order of the atomics does not matter), the second over tiles of 64 x 128
// elements, encoded along their rows from registers and along their columns through shared memory.
// HBM bounds both: (2 or 4) R C bytes in, 9/16 R C out per form.
#include <type_traits>

#include "ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTileR = 64, kTileC = 128;  // elements of a tile of the two-form kernel

__host__ __device__ inline int64_t pad_to(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

__device__ __forceinline__ float elem(float v) { return v; }
__device__ __forceinline__ float elem(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem(__half v) { return __half2float(v); }

// N consecutive elements from p as fp32; those at or past `live` are zero.  wide: p is 16-byte aligned.
template <int N, typename T>
__device__ __forceinline__ void load_row(const T* p, int64_t live, bool wide, float (&v)[N]) {
    constexpr int per = 16 / (int)sizeof(T);
    if (wide && live >= N) {
#pragma unroll
        for (int i = 0; i < N / per; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
            const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
            for (int j = 0; j < per; ++j) v[per * i + j] = elem(e[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < live ? elem(p[i]) : 0.f;
    }
}

__device__ __forceinline__ float row_scale(float amax) {
    const float g = __fdiv_rn(amax, 2688.f);
    return g == 0.f ? 1.f : g;
}

// One block of 16 elements under the row scale g: two words of codes; returns the scale byte.
__device__ __forceinline__ uint32_t encode_block(float* v, float g, bool given, uint32_t& c0, uint32_t& c1) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
    const uint32_t sb = f32_to_e4m3_sat(__fdiv_rn(__fdiv_rn(amax, g), 6.f));
    const float D = __fmul_rn(e4m3x2_to_f2(sb).x, g);
    c0 = c1 = 0u;
    if (D == 0.f) return sb;
    if (given) {  // a row scale that is not the row's own may leave quotients far above 6: they saturate
        const float lim = 8.f * D;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = fminf(fmaxf(v[i], -lim), lim);
    }
    if (D >= 8.6736174e-19f && D <= 1.1529215e18f) {
        const float y = __frcp_rn(D);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float q0 = __fmul_rn(v[i], y);
            v[i] = __fmaf_rn(__fmaf_rn(-q0, D, v[i]), y, q0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(v[i], D);
    }
    c0 = e2m1x8_encode(v);
    c1 = e2m1x8_encode(v + 8);
    return sb;
}

// 32 elements (two blocks): 16 bytes of codes, two scale bytes.
__device__ __forceinline__ uint32_t encode_unit(float (&v)[32], float g, bool given, uint4& codes) {
    const uint32_t s0 = encode_block(v, g, given, codes.x, codes.y);
    const uint32_t s1 = encode_block(v + 16, g, given, codes.z, codes.w);
    return s0 | (s1 << 8);
}

// ------------------------------------------------------------------ row form
// `tpr` threads (32 .. 256) share a row; thread c of them the 32-element units c, c + tpr, ...
template <typename T>
__global__ void __launch_bounds__(kThreads)
    nvfp4_rows_kernel(const T* __restrict__ x, int64_t R, int64_t K, int64_t ld, bool wide, int tpr, uint8_t* __restrict__ q,
                      uint8_t* __restrict__ s, float* __restrict__ gs, bool given, bool gs_rows) {
    __shared__ float part[kThreads / 32];
    pdl_launch_dependents();  // a product launched behind this call fetches its weights meanwhile
    const int in_row = threadIdx.x % tpr, rows = kThreads / tpr;
    const int64_t r = (int64_t)blockIdx.x * rows + threadIdx.x / tpr;
    const int64_t Kp = pad_to(K, 256);
    const int units = (int)(Kp / 32);
    const bool live = r < R;
    const T* row = x + (live ? r : 0) * ld;
    float v[32];
    float g = 1.f;
    const int64_t u0 = in_row;
    if (live && u0 < units) load_row<32>(row + 32 * u0, K - 32 * u0, wide, v);
    if (!given) {
        float amax = 0.f;
        if (live && u0 < units) {
#pragma unroll
            for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(v[i]));
            float o[32];
            for (int64_t u = u0 + tpr; u < units; u += tpr) {
                load_row<32>(row + 32 * u, K - 32 * u, wide, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(o[i]));
            }
        }
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        if (tpr > 32) {
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
            __syncthreads();
            const int w0 = (threadIdx.x / tpr) * (tpr / 32);
            for (int w = 0; w < tpr / 32; ++w) amax = fmaxf(amax, part[w0 + w]);
        }
        g = row_scale(amax);
        if (live && in_row == 0) gs[r] = g;
    } else if (live) {
        g = gs[gs_rows ? r : 0];
    }
    for (int64_t u = u0; live && u < units; u += tpr) {
        if (u != u0) load_row<32>(row + 32 * u, K - 32 * u, wide, v);
        uint4 codes;
        const uint32_t sb = encode_unit(v, g, given, codes);
        *reinterpret_cast<uint4*>(q + mma_tile_offset(r, u, Kp)) = codes;
        *reinterpret_cast<uint16_t*>(s + mma_scale_offset(r, 2 * u, 2 * Kp)) = (uint16_t)sb;
    }
}

// ------------------------------------------------------------------ both forms
// Maxima of |x| over rows and columns as fp32 bits in row_max[R] and col_max[C] (zeroed before).  A CTA
// takes 256 columns x 256 rows: warp w the rows 32 w ..., lane l the columns 8 l ...
template <typename T>
__global__ void __launch_bounds__(kThreads)
    nvfp4_maxima_kernel(const T* __restrict__ x, int64_t R, int64_t C, int64_t ld, bool wide, int col_tiles,
                        unsigned* __restrict__ row_max, unsigned* __restrict__ col_max) {
    __shared__ float part[kThreads / 32][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
    const int64_t c0 = ct * 256 + 8 * lane, r0 = rt * 256 + 32 * warp;
    float cm[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cm[i] = 0.f;
    unsigned mine = 0;
#pragma unroll 4
    for (int j = 0; j < 32; ++j) {
        float v[8];
        float m = 0.f;
        if (r0 + j < R && c0 < C) {
            load_row<8>(x + (r0 + j) * ld + c0, C - c0, wide, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cm[i] = fmaxf(cm[i], fabsf(v[i]));
                m = fmaxf(m, fabsf(v[i]));
            }
        }
        const unsigned rm = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (lane == j) mine = rm;
    }
    if (row_max && r0 + lane < R) atomicMax(row_max + r0 + lane, mine);
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][8 * lane + i] = cm[i];
    __syncthreads();
    float m = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, part[w][threadIdx.x]);
    const int64_t c = ct * 256 + threadIdx.x;
    if (c < C) atomicMax(col_max + c, __float_as_uint(m));
}

// A tile of 64 rows x 128 columns of x: thread (r, j) encodes 32 elements of row r for the row form, and
// thread (c, j) 32 elements of column c, through shared memory, for the column form.  Tiles cover the
// padded contractions (256 multiples), whose padding is written as zeros.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    nvfp4_both_kernel(const T* __restrict__ x, int64_t R, int64_t C, int64_t ld, bool wide, int col_tiles,
                      const unsigned* __restrict__ row_max, const unsigned* __restrict__ col_max, moe_nvfp4_operand rows,
                      moe_nvfp4_operand cols, bool given) {
    __shared__ T tile[kTileR][kTileC + 16 / sizeof(T)];
    const int64_t r0 = (int64_t)(blockIdx.x / col_tiles) * kTileR, c0 = (int64_t)(blockIdx.x % col_tiles) * kTileC;
    const int64_t Cp = pad_to(C, 256), Rp = pad_to(R, 256);
    {
        const int i = threadIdx.x >> 2, j = threadIdx.x & 3;
        const int64_t r = r0 + i, c = c0 + 32 * j;
        float v[32];
        load_row<32>(x + (r < R ? r : 0) * ld + c, r < R ? C - c : 0, wide, v);
#pragma unroll
        for (int m = 0; m < 32; ++m) {  // exact: v came from a T
            if constexpr (std::is_same<T, float>::value) tile[i][32 * j + m] = v[m];
            else if constexpr (std::is_same<T, __half>::value) tile[i][32 * j + m] = __float2half_rn(v[m]);
            else tile[i][32 * j + m] = __float2bfloat16_rn(v[m]);
        }
        if (rows.q && r < R && c < Cp) {
            const float g = given ? rows.gs[rows.gs_rows ? r : 0] : row_scale(__uint_as_float(__ldg(row_max + r)));
            if (!given && c == 0) rows.gs[r] = g;
            uint4 codes;
            const uint32_t sb = encode_unit(v, g, given, codes);
            *reinterpret_cast<uint4*>(rows.q + mma_tile_offset(r, c / 32, Cp)) = codes;
            *reinterpret_cast<uint16_t*>(rows.s + mma_scale_offset(r, c / 16, 2 * Cp)) = (uint16_t)sb;
        }
    }
    __syncthreads();
    {
        const int i = threadIdx.x & 127, j = threadIdx.x >> 7;
        const int64_t c = c0 + i, r = r0 + 32 * j;
        if (c >= C || r >= Rp) return;
        float v[32];
#pragma unroll
        for (int m = 0; m < 32; ++m) v[m] = elem(tile[32 * j + m][i]);
        const float g = given ? cols.gs[cols.gs_rows ? c : 0] : row_scale(__uint_as_float(__ldg(col_max + c)));
        if (!given && r == 0) cols.gs[c] = g;
        uint4 codes;
        const uint32_t sb = encode_unit(v, g, given, codes);
        *reinterpret_cast<uint4*>(cols.q + mma_tile_offset(c, r / 32, Rp)) = codes;
        *reinterpret_cast<uint16_t*>(cols.s + mma_scale_offset(c, r / 16, 2 * Rp)) = (uint16_t)sb;
    }
}

template <typename T>
cudaError_t quantize(const T* x, int64_t R, int64_t C, int64_t ld, const moe_nvfp4_operand* rows,
                     const moe_nvfp4_operand* cols, bool given, unsigned* maxima, cudaStream_t st, bool pdl) {
    bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
    if (!cols) {
        const int64_t units = pad_to(C, 256) / 32;
        int tpr = 32;
        while (tpr < kThreads && tpr < units) tpr *= 2;
        const int64_t per = kThreads / tpr, blocks = (R + per - 1) / per;
        bool gr = rows->gs_rows != 0;
        uint8_t *q = rows->q, *s = rows->s;
        float* gs = rows->gs;
        void* args[] = {&x, &R, &C, &ld, &wide, &tpr, &q, &s, &gs, &given, &gr};
        return launch_kernel((const void*)nvfp4_rows_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), 0, st, pdl, args);
    }
    unsigned* row_max = rows ? maxima : nullptr;
    unsigned* col_max = maxima + (rows ? R : 0);
    if (!given) {
        cudaError_t e = cudaMemsetAsync(maxima, 0, sizeof(unsigned) * (size_t)((rows ? R : 0) + C), st);
        if (e != cudaSuccess) return e;
        int ct = (int)((C + 255) / 256);
        void* args[] = {&x, &R, &C, &ld, &wide, &ct, &row_max, &col_max};
        e = launch_kernel((const void*)nvfp4_maxima_kernel<T>, dim3((unsigned)(ct * ((R + 255) / 256))), dim3(kThreads), 0, st,
                          false, args);
        if (e != cudaSuccess) return e;
    }
    // the padded contractions: columns to 256 for the row form, rows to 256 for the column form
    int ct = (int)(pad_to(C, rows ? 256 : kTileC) / kTileC);
    const int64_t rt = pad_to(R, 256) / kTileR;
    moe_nvfp4_operand a = rows ? *rows : moe_nvfp4_operand{nullptr, nullptr, nullptr, 0}, b = *cols;
    void* args[] = {&x, &R, &C, &ld, &wide, &ct, &row_max, &col_max, &a, &b, &given};
    return launch_kernel((const void*)nvfp4_both_kernel<T>, dim3((unsigned)(ct * rt)), dim3(kThreads), 0, st, false, args);
}

// Values of an operand: (E2M1 * E4M3) * row scale, the exact product of the first two rounded once.
__global__ void __launch_bounds__(kThreads)
    nvfp4_values_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, const float* __restrict__ gs, bool gs_rows,
                        int64_t R, int64_t K, float* __restrict__ v) {
    const int64_t units = (K + 31) / 32, Kp = pad_to(K, 256);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < R * units; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / units, u = i % units;
        const uint4 c = *reinterpret_cast<const uint4*>(q + mma_tile_offset(r, u, Kp));
        const float2 sc = e4m3x2_to_f2(*reinterpret_cast<const uint16_t*>(s + mma_scale_offset(r, 2 * u, 2 * Kp)));
        const float g = gs[gs_rows ? r : 0];
        const uint32_t words[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            uint32_t h[4];
            e2m1x8_to_h2(words[m], h);
            const float sv = m < 2 ? sc.x : sc.y;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 p = h2_to_f2(h[j / 2]);
                const int64_t k = 32 * u + 8 * m + j;
                if (k < K) v[r * K + k] = __fmul_rn(__fmul_rn(j & 1 ? p.y : p.x, sv), g);
            }
        }
    }
}

}  // namespace

cudaError_t launch_nvfp4_quantize(const void* x, moe_dtype dtype, int64_t R, int64_t C, int64_t ld,
                                  const moe_nvfp4_operand* rows, const moe_nvfp4_operand* cols, bool given, void* maxima,
                                  cudaStream_t st, bool pdl) {
    if (R == 0 || C == 0) return cudaSuccess;
    unsigned* m = static_cast<unsigned*>(maxima);
    if (dtype == MOE_F32) return quantize(static_cast<const float*>(x), R, C, ld, rows, cols, given, m, st, pdl);
    if (dtype == MOE_BF16) return quantize(static_cast<const __nv_bfloat16*>(x), R, C, ld, rows, cols, given, m, st, pdl);
    return quantize(static_cast<const __half*>(x), R, C, ld, rows, cols, given, m, st, pdl);
}

cudaError_t launch_nvfp4_values(const moe_nvfp4_operand* op, int64_t R, int64_t K, float* v, cudaStream_t st) {
    if (R == 0 || K == 0) return cudaSuccess;
    const int64_t n = R * ((K + 31) / 32);
    int64_t blocks = (n + kThreads - 1) / kThreads;
    if (blocks > 152 * 64) blocks = 152 * 64;
    nvfp4_values_kernel<<<(unsigned)blocks, kThreads, 0, st>>>(op->q, op->s, op->gs, op->gs_rows != 0, R, K, v);
    return cudaGetLastError();
}

}  // namespace moe
