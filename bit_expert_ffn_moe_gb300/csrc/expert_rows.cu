// expert_rows.cu -- token rows on their way to the experts and back.  r(t,j) = inv[t k + j] is the row of token t's slot j in
// expert order (an entry outside [0, T k): none), w the routing weights (null: ones):
//   spread   rows[r(t,j)] = w[t][j] x[t]                        tokens to experts; the gradient of the experts' outputs
//   gather   y[t] = sum_j w[t][j] rows[r(t,j)]                  experts to tokens; the gradient of the tokens
//   spread and gather with the weights' gradient, dw[t][j] = <a[t], b[r(t,j)]>, in the same pass over b
// One product or one fp32 sum in the order of the slots, rounded once to the rows' type.  Nothing is read twice but inv and w, so all
// are bound by HBM: (1 + k) T d elements, (1 + 2 k) T d for the spread with dw.
// Rows are moved in pieces of 16 bytes where every matrix allows it (addresses, strides and d), else in words: two 16-bit
// elements, from one word or (in rows that start between two words) from two.
#include "ops.cuh"
#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// WORDS words of a row: its elements e .. e + N - 1.  WORDS = 4: aligned; 1: 16-bit elements may begin in the middle of a word, and the
// last one of a row may be alone.
template <typename T, int WORDS>
struct Piece {
    static constexpr int N = WORDS * 4 / (int)sizeof(T);
    static constexpr bool kHalves = WORDS == 1 && sizeof(T) == 2;
    uint32_t w[kHalves ? 2 : WORDS];

    // Where in a word the pieces of a row begin, in bits (they begin at even elements).
    __device__ __forceinline__ static uint32_t shift_of(const T* row) {
        if constexpr (kHalves) return (uint32_t)(reinterpret_cast<uintptr_t>(row) & 2) * 8;
        else return 0;
    }

    // (All slots' loads stand in front of their uses, so that several are in flight instead of each waiting next to its use: 90 us for the
    // gather of 4096 tokens of 8 slots of 8192 features, where loads in a loop with their uses took 297.)
    __device__ __forceinline__ void load(const T* row, int e, int d) {
        const T* p = row + e;
        if constexpr (WORDS == 4) {
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
        } else if constexpr (!kHalves) {
            asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
        } else {
            // the word that the piece begins in (which is in the allocation with it), and where it begins in its middle the next one
            const uintptr_t at = reinterpret_cast<uintptr_t>(p);
            w[1] = 0;
            asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w[0]) : "l"(at & ~(uintptr_t)3));
            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}"
                         : "+r"(w[1])
                         : "l"((at & ~(uintptr_t)3) + 4), "r"(e + 1 < d ? (uint32_t)(at & 2) : 0u));
        }
    }
    // Once loaded: the words as they would be in a row that begins with a word.
    __device__ __forceinline__ void settle(uint32_t shift) {
        if constexpr (kHalves) w[0] = __funnelshift_r(w[0], w[1], shift);
    }
    __device__ __forceinline__ void store(T* row, int e, int d) const {
        T* p = row + e;
        if constexpr (WORDS == 4) {
            __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        } else if (!kHalves || (reinterpret_cast<uintptr_t>(p) % 4 == 0 && e + 1 < d)) {
            *reinterpret_cast<uint32_t*>(p) = w[0];
        } else {
            reinterpret_cast<uint16_t*>(p)[0] = (uint16_t)w[0];
            if (e + 1 < d) reinterpret_cast<uint16_t*>(p)[1] = (uint16_t)(w[0] >> 16);
        }
    }
    __device__ __forceinline__ void get(float (&f)[N]) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                const float2 v = unpack<T>(w[i]);
                f[2 * i] = v.x, f[2 * i + 1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
            else w[i] = pack<T>(f[2 * i], f[2 * i + 1]);
        }
    }
    __device__ __forceinline__ Piece scaled(float s) const {
        float f[N];
        get(f);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] *= s;
        Piece r;
        r.set(f);
        return r;
    }
};

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

// One thread per piece of 16 bytes of a token's row; SPREAD: loaded once and stored k times, else loaded k times (eight in flight)
// and stored once.
template <typename T, bool SPREAD>
__global__ void __launch_bounds__(kThreads) move_kernel(const MoveArgs m) {
    using P = Piece<T, 4>;
    pdl_wait();
    pdl_launch_dependents();
    const int pieces = m.d / P::N;
    const int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t t = (q >> 32) == 0 ? (int64_t)((uint32_t)q / (uint32_t)pieces) : q / pieces;
    if (t >= m.T) return;
    const int e = (int)(q - t * pieces) * P::N;
    if constexpr (SPREAD) {
        P x;
        x.load(static_cast<const T*>(m.a) + t * m.lda, e, m.d);
#pragma unroll 8
        for (int j = 0; j < m.k; ++j) {
            const int r = row_of(m, t * m.k + j);
            if (r < 0) continue;
            T* to = static_cast<T*>(m.out) + r * m.ldo;
            if (m.w) x.scaled(__ldg(m.w + t * m.k + j)).store(to, e, m.d);
            else x.store(to, e, m.d);
        }
    } else {
        float sum[P::N] = {};
        for (int j0 = 0; j0 < m.k; j0 += 8) {
            P b[8];
            int r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = j0 + j < m.k ? row_of(m, t * m.k + j0 + j) : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j)  // (a slot without a row loads row 0 and leaves it out)
                if (j0 + j < m.k) b[j].load(static_cast<const T*>(m.b) + max(r[j], 0) * m.ldb, e, m.d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j0 + j >= m.k) break;
                const float w = m.w ? __ldg(m.w + t * m.k + j0 + j) : 1.f;
                float f[P::N];
                b[j].get(f);
#pragma unroll
                for (int i = 0; i < P::N; ++i) sum[i] = r[j] >= 0 ? fmaf(w, f[i], sum[i]) : sum[i];
            }
        }
        P y;
        y.set(sum);
        y.store(static_cast<T*>(m.out) + t * m.ldo, e, m.d);
    }
}

// `warps` warps of a CTA share a token, whose rows' places are in registers; PIECES pieces a thread of its row and of all its slots
// (k <= SLOTS) are in flight at a time.  DW: with the weights' gradient.
template <typename T, int WORDS, bool SPREAD, bool DW, int SLOTS, int PIECES>
__global__ void __launch_bounds__(kThreads, SLOTS <= 8 ? 3 : SLOTS <= 16 ? 2 : 1) token_kernel(const MoveArgs m, const int warps) {
    using P = Piece<T, WORDS>;
    __shared__ float part[kThreads / 32][SLOTS];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tokens = kThreads / 32 / warps, mine = warp / warps;
    const int64_t t = (int64_t)blockIdx.x * tokens + mine;
    const bool live = t < m.T;
    const int first = threadIdx.x - mine * warps * 32, step = warps * 32 * P::N, d = m.d, k = m.k;
    const T* const arow = static_cast<const T*>(m.a) + t * m.lda;
    const uint32_t a_shift = P::shift_of(arow);
    int r[SLOTS];
    uint32_t b_shift[SLOTS];
    float w[SLOTS], acc[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        r[j] = live && j < k ? row_of(m, t * k + j) : -1;
        w[j] = r[j] >= 0 && m.w ? __ldg(m.w + t * k + j) : 1.f;
        b_shift[j] = P::shift_of(static_cast<const T*>(m.b) + r[j] * m.ldb);
        acc[j] = 0.f;
    }
    if (live)
        for (uint32_t e0 = first * P::N; e0 < (uint32_t)d; e0 += PIECES * step) {  // (unsigned: rows of up to 2^31 - 1 elements)
            P a[PIECES], b[PIECES][SLOTS];
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                const int e = (int)min(e0 + q * step, (uint32_t)((d - 1) / P::N * P::N));  // (behind the end: the last piece again)
                if (SPREAD || DW) a[q].load(arow, e, d);
                if (!SPREAD || DW)
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j)
                        if (r[j] >= 0) b[q][j].load(static_cast<const T*>(m.b) + r[j] * m.ldb, e, d);
            }
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                if (PIECES > 1 && e0 + q * step >= (uint32_t)d) break;
                const int e = (int)(e0 + q * step);
                float fa[P::N], sum[P::N] = {};
                if (SPREAD || DW) a[q].settle(a_shift), a[q].get(fa);
#pragma unroll
                for (int j = 0; j < SLOTS; ++j) {
                    if (r[j] < 0) continue;
                    float fb[P::N];
                    if (!SPREAD || DW) b[q][j].settle(b_shift[j]), b[q][j].get(fb);
#pragma unroll
                    for (int i = 0; i < P::N; ++i) {
                        if (DW && (WORDS == 4 || e + i < d)) acc[j] = fmaf(fa[i], fb[i], acc[j]);
                        if (!SPREAD) sum[i] = fmaf(w[j], fb[i], sum[i]);
                    }
                    if (SPREAD && m.out) {
                        T* to = static_cast<T*>(m.out) + r[j] * m.ldo;
                        if (m.w) a[q].scaled(w[j]).store(to, e, d);
                        else a[q].store(to, e, d);
                    }
                }
                if (!SPREAD && m.out) {
                    P y;
                    y.set(sum);
                    y.store(static_cast<T*>(m.out) + t * m.ldo, e, d);
                }
            }
        }
    if (!DW) return;
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

template <typename T, int WORDS, bool SPREAD, bool DW, int SLOTS, int PIECES>
cudaError_t launch_token(MoveArgs m, cudaStream_t st) {
    const int64_t pieces = ((int64_t)m.d + Piece<T, WORDS>::N * PIECES - 1) / (Piece<T, WORDS>::N * PIECES);
    int warps = 1;
    while (warps < kThreads / 32 && warps * 32 < pieces) warps *= 2;
    const int tokens = kThreads / 32 / warps;
    void* args[] = {&m, &warps};
    return launch_kernel((const void*)token_kernel<T, WORDS, SPREAD, DW, SLOTS, PIECES>, dim3((m.T + tokens - 1) / tokens), dim3(kThreads), 0,
                         st, true, args);
}
template <typename T, int WORDS, bool SPREAD, bool DW>
cudaError_t launch_slots(const MoveArgs& m, cudaStream_t st) {
    constexpr int kMore = WORDS == 1 && (!DW || sizeof(T) == 4) ? 2 : 1;  // words: more of them in flight
    if (m.k <= 1) return launch_token<T, WORDS, SPREAD, DW, 1, 4>(m, st);
    if (m.k <= 2) return launch_token<T, WORDS, SPREAD, DW, 2, 2 * kMore>(m, st);
    if (m.k <= 4) return launch_token<T, WORDS, SPREAD, DW, 4, 2 * kMore>(m, st);
    if (m.k <= 6) return launch_token<T, WORDS, SPREAD, DW, 6, kMore>(m, st);
    if (m.k <= 8) return launch_token<T, WORDS, SPREAD, DW, 8, kMore>(m, st);
    if (m.k <= 12) return launch_token<T, WORDS, SPREAD, DW, 12, 1>(m, st);
    if (m.k <= 16) return launch_token<T, WORDS, SPREAD, DW, 16, 1>(m, st);
    return launch_token<T, WORDS, SPREAD, DW, 32, 1>(m, st);
}

template <typename T, bool SPREAD>
cudaError_t launch_type(MoveArgs m, cudaStream_t st) {
    constexpr int N = 16 / (int)sizeof(T);
    auto wide = [&](const void* p, int64_t ld) { return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % N == 0); };
    const bool pieces = m.d % N == 0 && wide(m.a, m.lda) && wide(m.b, m.ldb) && wide(m.out, m.ldo);
    if (m.dw) return pieces ? launch_slots<T, 4, SPREAD, true>(m, st) : launch_slots<T, 1, SPREAD, true>(m, st);
    if (!pieces) return launch_slots<T, 1, SPREAD, false>(m, st);
    // (4096 x 8 x 8192: 116 us with a thread per piece, 90 with warps per token; 4 x 8 x 8192: 2.6 and 5)
    if (!SPREAD && m.T >= 2 * sm_count() && m.d / N >= 64) return launch_slots<T, 4, SPREAD, false>(m, st);
    const int64_t blocks = ((int64_t)m.T * (m.d / N) + kThreads - 1) / kThreads;
    void* args[] = {&m};
    return launch_kernel((const void*)move_kernel<T, SPREAD>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, args);
}

}  // namespace

cudaError_t launch_expert_rows(bool spread, moe_dtype dtype, const void* a, int64_t lda, const void* b, int64_t ldb, void* out,
                               int64_t ldo, const int32_t* inv, const float* w, float* dw, int T, int k, int d, cudaStream_t st) {
    const MoveArgs m = {a, lda, b, ldb, out, ldo, inv, w, dw, T, k, d};
    switch (dtype) {
        case MOE_F32: return spread ? launch_type<float, true>(m, st) : launch_type<float, false>(m, st);
        case MOE_BF16: return spread ? launch_type<__nv_bfloat16, true>(m, st) : launch_type<__nv_bfloat16, false>(m, st);
        default: return spread ? launch_type<__half, true>(m, st) : launch_type<__half, false>(m, st);
    }
}

}  // namespace moe
