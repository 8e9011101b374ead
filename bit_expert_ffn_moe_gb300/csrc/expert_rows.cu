// expert_rows.cu -- token rows on their way to the experts and back.  r(t,j) = inv[t k + j] is the row of token t's slot j in
// expert order (an entry outside [0, T k): none), w the routing weights (null: ones):
//   spread   rows[r(t,j)] = w[t][j] x[t]                        tokens to experts; the gradient of the experts' outputs
//   gather   y[t] = sum_j w[t][j] rows[r(t,j)]                  experts to tokens; the gradient of the tokens
//   spread and gather with the weights' gradient, dw[t][j] = <a[t], b[r(t,j)]>, in the same pass over b
// One product or one fp32 sum in the order of the slots, rounded once to the rows' type.  Nothing is read twice but inv and w, so all
// are bound by HBM: (1 + k) T d elements, (1 + 2 k) T d for the spread with dw.
// Rows are moved in pieces of 16 bytes where every matrix allows it (addresses, strides and d), else element by element.
#include "ops.cuh"
#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements, loaded and stored at once.
template <typename T, int N>
struct alignas(sizeof(T) * N) Piece {
    T v[N];
};
template <typename T, int N>
__device__ __forceinline__ Piece<T, N> load(const T* p) {
    Piece<T, N> r;
    if constexpr (sizeof(T) * N == 16) *reinterpret_cast<uint4*>(&r) = __ldcs(reinterpret_cast<const uint4*>(p));
    else r.v[0] = *p;
    return r;
}
template <typename T, int N>
__device__ __forceinline__ void store(T* p, const Piece<T, N>& r) {
    if constexpr (sizeof(T) * N == 16) __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&r));
    else *p = r.v[0];
}
template <typename T, int N>
__device__ __forceinline__ Piece<T, N> scaled(const Piece<T, N>& a, float w) {
    Piece<T, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(w * to_f32(a.v[i]));
    return r;
}

struct MoveArgs {
    const void* a;  // [T] rows: x, dy
    int64_t lda;
    const void* b;  // [T k] rows, read
    int64_t ldb;
    void* out;  // spread: [T k] rows; gather: [T] rows
    int64_t ldo;
    const int32_t* inv;
    const float* w;  // or null
    float* dw;
    int T, k, d;
};

__device__ __forceinline__ int row_of(const MoveArgs& m, int64_t pair) {
    const int r = __ldg(m.inv + pair);
    return (unsigned)r < (unsigned)(m.T * m.k) ? r : -1;
}

// One thread per piece of a token's row; SPREAD: loaded once and stored k times, else loaded k times (eight in flight) and
// stored once.
template <typename T, int N, bool SPREAD>
__global__ void __launch_bounds__(kThreads) move_kernel(const MoveArgs m) {
    pdl_wait();
    pdl_launch_dependents();
    const int pieces = m.d / N;
    const int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t t = (q >> 32) == 0 ? (int64_t)((uint32_t)q / (uint32_t)pieces) : q / pieces;
    if (t >= m.T) return;
    const int64_t c = (q - t * pieces) * N;
    if constexpr (SPREAD) {
        const Piece<T, N> x = load<T, N>(static_cast<const T*>(m.a) + t * m.lda + c);
#pragma unroll 8
        for (int j = 0; j < m.k; ++j) {
            const int r = row_of(m, t * m.k + j);
            if (r < 0) continue;
            store<T, N>(static_cast<T*>(m.out) + r * m.ldo + c, m.w ? scaled(x, __ldg(m.w + t * m.k + j)) : x);
        }
    } else {
        float sum[N] = {};
        for (int j0 = 0; j0 < m.k; j0 += 8) {
            Piece<T, N> b[8];
            int r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[j] = j0 + j < m.k ? row_of(m, t * m.k + j0 + j) : -1;
                if (r[j] >= 0) b[j] = load<T, N>(static_cast<const T*>(m.b) + r[j] * m.ldb + c);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (r[j] < 0) continue;
                const float w = m.w ? __ldg(m.w + t * m.k + j0 + j) : 1.f;
#pragma unroll
                for (int i = 0; i < N; ++i) sum[i] = fmaf(w, to_f32(b[j].v[i]), sum[i]);
            }
        }
        Piece<T, N> y;
#pragma unroll
        for (int i = 0; i < N; ++i) y.v[i] = from_f32<T>(sum[i]);
        store<T, N>(static_cast<T*>(m.out) + t * m.ldo + c, y);
    }
}

// With dw: `warps` warps of a CTA share a token; the pieces of all its slots (k <= SLOTS) are in registers at a time, with its own.
template <typename T, int N, bool SPREAD, int SLOTS>
__global__ void __launch_bounds__(kThreads, SLOTS <= 8 ? 3 : 1) move_dw_kernel(const MoveArgs m, const int warps) {
    __shared__ float part[kThreads / 32][SLOTS];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tokens = kThreads / 32 / warps, mine = warp / warps;
    const int64_t t = (int64_t)blockIdx.x * tokens + mine;
    const bool live = t < m.T;
    const int first = threadIdx.x - mine * warps * 32, step = warps * 32, pieces = m.d / N, k = m.k;
    int r[SLOTS];
    float w[SLOTS], acc[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        r[j] = live && j < k ? row_of(m, t * k + j) : -1;
        w[j] = r[j] >= 0 && m.w ? __ldg(m.w + t * k + j) : 1.f;
        acc[j] = 0.f;
    }
    if (live)
        for (int c = first; c < pieces; c += step) {
            const Piece<T, N> a = load<T, N>(static_cast<const T*>(m.a) + t * m.lda + (int64_t)c * N);
            Piece<T, N> b[SLOTS];
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
                if (r[j] >= 0) b[j] = load<T, N>(static_cast<const T*>(m.b) + r[j] * m.ldb + (int64_t)c * N);
            float sum[N] = {};
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                if (r[j] < 0) continue;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float v = to_f32(b[j].v[i]);
                    acc[j] = fmaf(to_f32(a.v[i]), v, acc[j]);
                    if constexpr (!SPREAD) sum[i] = fmaf(w[j], v, sum[i]);
                }
                if (SPREAD && m.out)
                    store<T, N>(static_cast<T*>(m.out) + r[j] * m.ldo + (int64_t)c * N, m.w ? scaled(a, w[j]) : a);
            }
            if (!SPREAD && m.out) {
                Piece<T, N> y;
#pragma unroll
                for (int i = 0; i < N; ++i) y.v[i] = from_f32<T>(sum[i]);
                store<T, N>(static_cast<T*>(m.out) + t * m.ldo + (int64_t)c * N, y);
            }
        }
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        acc[j] = warp_butterfly_sum(acc[j]);
        if (lane == 0) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (live && warp % warps == 0 && lane < k) {
        float sum = 0.f;
        for (int v = 0; v < warps; ++v) sum += part[warp + v][lane];
        m.dw[t * k + lane] = sum;
    }
}

template <typename T, int N, bool SPREAD>
cudaError_t launch_move(MoveArgs m, cudaStream_t st) {
    const int pieces = m.d / N;
    if (!m.dw) {
        const int64_t blocks = ((int64_t)m.T * pieces + kThreads - 1) / kThreads;
        void* args[] = {&m};
        return launch_kernel((const void*)move_kernel<T, N, SPREAD>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, args);
    }
    int warps = 1;
    while (warps < kThreads / 32 && warps * 32 < pieces) warps *= 2;
    const int tokens = kThreads / 32 / warps;
    const void* f = m.k <= 2   ? (const void*)move_dw_kernel<T, N, SPREAD, 2>
                    : m.k <= 4 ? (const void*)move_dw_kernel<T, N, SPREAD, 4>
                    : m.k <= 8 ? (const void*)move_dw_kernel<T, N, SPREAD, 8>
                    : m.k <= 16 ? (const void*)move_dw_kernel<T, N, SPREAD, 16>
                                : (const void*)move_dw_kernel<T, N, SPREAD, 32>;
    void* args[] = {&m, &warps};
    return launch_kernel(f, dim3((m.T + tokens - 1) / tokens), dim3(kThreads), 0, st, true, args);
}

template <typename T>
cudaError_t launch_type(const MoveArgs& m, bool spread, cudaStream_t st) {
    constexpr int N = 16 / (int)sizeof(T);
    auto wide = [&](const void* p, int64_t ld) { return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % N == 0); };
    if (m.d % N == 0 && wide(m.a, m.lda) && wide(m.b, m.ldb) && wide(m.out, m.ldo))
        return spread ? launch_move<T, N, true>(m, st) : launch_move<T, N, false>(m, st);
    return spread ? launch_move<T, 1, true>(m, st) : launch_move<T, 1, false>(m, st);
}

}  // namespace

cudaError_t launch_expert_rows(bool spread, moe_dtype dtype, const void* a, int64_t lda, const void* b, int64_t ldb, void* out,
                               int64_t ldo, const int32_t* inv, const float* w, float* dw, int T, int k, int d, cudaStream_t st) {
    const MoveArgs m = {a, lda, b, ldb, out, ldo, inv, w, dw, T, k, d};
    switch (dtype) {
        case MOE_F32: return launch_type<float>(m, spread, st);
        case MOE_BF16: return launch_type<__nv_bfloat16>(m, spread, st);
        default: return launch_type<__half>(m, spread, st);
    }
}

}  // namespace moe
