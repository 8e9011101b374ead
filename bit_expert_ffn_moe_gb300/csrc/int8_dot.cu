// int8_dot.cu -- the 8-bit products of few rows: dot products of four bytes (dp4a), the weights read once.
// The weight rows of all active experts' matrices are dealt out evenly to the CTAs, so that no partial sums have to be exchanged.
// A warp takes pieces of 32 weight rows x 128 values (eight 16-byte loads a lane) in turn, the next one's loads in flight while it
// works on one, and adds its sums to the rows' in shared memory: sums of whole numbers, so their order does not matter.
// Rows of x that are not an operand yet are quantised by every CTA for itself, while its first weights are on their way.
// Bound by the weight read: 1 x 4096 x 8192 (33.6 MB) 10.2 us, 11.3 with the quantisation of x; 8 experts of 4096 x 8192 (268 MB) 47.9 us, 5.6 TB/s.
#include "int8_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kTokens = 4;   // activation rows at a time
constexpr int kRows = 512;   // weight rows at a time
constexpr int kK = kInt8DotK;

// Four fp16 whole numbers as four bytes.
__device__ __forceinline__ uint32_t bytes_of(uint2 h) {
    const __half2 a = *reinterpret_cast<const __half2*>(&h.x), b = *reinterpret_cast<const __half2*>(&h.y);
    return (uint32_t)(__half2int_rn(__low2half(a)) & 255) | ((uint32_t)(__half2int_rn(__high2half(a)) & 255) << 8) |
           ((uint32_t)(__half2int_rn(__low2half(b)) & 255) << 16) | ((uint32_t)(__half2int_rn(__high2half(b)) & 255) << 24);
}
__device__ __forceinline__ uint32_t bytes_of(const float* q) {
    return (uint32_t)(__float2int_rn(q[0]) & 255) | ((uint32_t)(__float2int_rn(q[1]) & 255) << 8) |
           ((uint32_t)(__float2int_rn(q[2]) & 255) << 16) | ((uint32_t)(__float2int_rn(q[3]) & 255) << 24);
}

struct Shared {
    uint8_t x[kTokens][kK];
    int acc[kTokens][kRows];
    float sx[kTokens];
    uint32_t most[kWarps];
    int active[kMaxE], n_active;
};

// Pieces of a block of weight rows: rows 32 g .. of the block, steps 2 c and 2 c + 1 of 64 values from k0 on.
struct Pieces {
    const uint8_t* w;  // the block's matrix
    int64_t n0;        // its first row
    int rows, KT, k0, per;  // rows; steps of a matrix row; the first step; pieces of 32 rows
};
struct At {
    int g, c;
};
__device__ __forceinline__ void advance(At& at, int by, int per) {
    at.c += by;
    while (at.c >= per) at.c -= per, ++at.g;
}
// Lane (i, j) = (lane % 8, lane / 8) loads the 16 bytes j of rows i, i + 8, i + 16, i + 24; zeros behind the rows and the last step.
__device__ __forceinline__ void load(const Pieces& p, const At& at, uint4 (&w)[2][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 32 * at.g + (lane & 7) + 8 * r;
        const int64_t n = p.n0 + row;
        const uint8_t* from = p.w + ((n >> 7) * p.KT + p.k0 + 2 * at.c) * kInt8Tile + (n & 127) * 16 + (lane >> 3) * 2048;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const bool there = row < p.rows && p.k0 + 2 * at.c + u < p.KT && at.c < p.per;
            w[u][r] = there ? ldg_stream(from + u * kInt8Tile) : make_uint4(0, 0, 0, 0);
        }
    }
}
template <int TM>
__device__ __forceinline__ void dot(Shared& s, const At& at, const uint4 (&w)[2][4]) {
    const int lane = threadIdx.x & 31;
    int acc[4][TM] = {};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const uint4 v = *reinterpret_cast<const uint4*>(&s.x[t][(2 * at.c + u) * 64 + (lane >> 3) * 16]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                acc[r][t] = __dp4a((int)w[u][r].x, (int)v.x, acc[r][t]);
                acc[r][t] = __dp4a((int)w[u][r].y, (int)v.y, acc[r][t]);
                acc[r][t] = __dp4a((int)w[u][r].z, (int)v.z, acc[r][t]);
                acc[r][t] = __dp4a((int)w[u][r].w, (int)v.w, acc[r][t]);
            }
        }
    // The sums over the four lanes of a row end in lane r of them for row i + 8 r (two exchanges of halves instead of four sums)
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const bool high = lane & 16, odd = lane & 8;
        const int a = (high ? acc[2][t] : acc[0][t]) + __shfl_xor_sync(0xffffffffu, high ? acc[0][t] : acc[2][t], 16);
        const int b = (high ? acc[3][t] : acc[1][t]) + __shfl_xor_sync(0xffffffffu, high ? acc[1][t] : acc[3][t], 16);
        const int v = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
        atomicAdd(&s.acc[t][32 * at.g + (lane & 7) + 16 * high + 8 * odd], v);
    }
}

template <typename T>
__device__ __forceinline__ void store(void* y, int64_t at, float v) { static_cast<T*>(y)[at] = int8_result<T>(v); }

// X: type of x, or void where it is an operand.  inv [a.M] (at most 32) or null: row r of the product is row p / k of x, where inv[p] = r.
template <typename X, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) int8_dot_kernel(const Int8ProductArgs a, const X* __restrict__ x, const int64_t ldx, const int32_t* __restrict__ inv, const int k,
                    const int y_dtype) {
    constexpr bool kQuantise = !__is_same(X, void);
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Shared& s = *reinterpret_cast<Shared*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int KT = (int)((a.K + 63) / 64);
    if (!a.early) pdl_wait(), pdl_launch_dependents();
    const int place = kQuantise && inv && lane < a.M ? __ldg(inv + lane) : -1;
    if (warp == 0) {  // the experts that have rows
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const bool has = e < a.E && (a.offsets ? int8_offset(a, e + 1) > int8_offset(a, e) : a.M > 0);
            const unsigned b = __ballot_sync(0xffffffffu, has);
            if (has) s.active[n + __popc(b & ((1u << lane) - 1u))] = e;
            n += __popc(b);
        }
        if (lane == 0) s.n_active = n;
    }
    for (int i = tid; i < kRows * kTokens; i += kThreads) (&s.acc[0][0])[i] = 0;
    __syncthreads();
    bool waited = !a.early;
    const int64_t NP = (a.N + 1) / 2, pairs = NP * s.n_active;  // weight rows are dealt out in twos
    const int64_t end = pairs * (blockIdx.x + 1) / gridDim.x;
    for (int64_t at = pairs * blockIdx.x / gridDim.x; at < end;) {
        const int e = s.active[at / NP];
        const int64_t n0 = 2 * (at % NP), n1 = min(min(a.N, n0 + 2 * (end - at)), n0 + kRows);
        at += (n1 - n0 + 1) / 2;
        const int64_t first = a.offsets ? int8_offset(a, e) : 0, count = a.offsets ? int8_offset(a, e + 1) - first : a.M;
        const int64_t row0 = a.offsets ? int8_first_row(first, e) : 0;
        for (int64_t t0 = 0; t0 < count; t0 += kTokens) {
            const int tokens = (int)min((int64_t)kTokens, count - t0);
            for (int k0 = 0; k0 < KT; k0 += kK / 64) {
                const int steps = min(KT - k0, kK / 64);
                const Pieces p = {a.w + (int64_t)e * int8_tiles(a.N, a.K) * kInt8Tile, n0, (int)(n1 - n0), KT, k0, (steps + 1) / 2};
                const int groups = (p.rows + 31) / 32;
                At now = {0, 0};
                advance(now, warp, p.per);
                uint4 w[2][4], next[2][4];
                if (now.g < groups) load(p, now, w);
                if (!waited) pdl_wait(), pdl_launch_dependents(), waited = true;
                if constexpr (kQuantise) {
                    // `share` warps a row
                    const int share = tokens == 1 ? kWarps : tokens == 2 ? kWarps / 2 : kWarps / 4, t = warp / share;
                    const int step = share * 32, c0 = tid - t * step, eights = 8 * steps;
                    int64_t from = first + t0 + t;
                    if (inv) from = max(__ffs(__ballot_sync(0xffffffffu, place == from)) - 1, 0) / k;
                    const X* row = x + from * ldx;
                    const bool wide = reinterpret_cast<uintptr_t>(row) % 16 == 0;
                    uint32_t most = 0;
                    auto get = [&](int c) {
                        Eight<X> v;
                        if (wide) v.template load<true>(row, 8 * (int64_t)c, a.K);
                        else v.template load<false>(row, 8 * (int64_t)c, a.K);
                        return v;
                    };
                    Eight<X> kept[2];
                    kept[0].clear(), kept[1].clear();
                    if (t < tokens) {
                        if (c0 < eights) kept[0] = get(c0);
                        if (c0 + step < eights) kept[1] = get(c0 + step);
                        most = kept[1].most(kept[0].most(0));
                        for (int c = c0 + 2 * step; c < eights; c += step) most = get(c).most(most);
                    }
                    most = __reduce_max_sync(0xffffffffu, Eight<X>::as_fp32(most));
                    if (lane == 0) s.most[warp] = most;
                    __syncthreads();
                    for (int i = 0; i < share; ++i) most = max(most, s.most[warp / share * share + i]);
                    const Scale sc = scale_of(most);
                    if (t < tokens) {
                        if (c0 == 0) s.sx[t] = sc.s;
                        auto put = [&](int c, const Eight<X>& v8) {
                            float v[8], q[8];
                            v8.get(v);
                            whole8(v, sc, q);
                            *reinterpret_cast<uint2*>(&s.x[t][8 * c]) = make_uint2(bytes_of(q), bytes_of(q + 4));
                        };
                        if (c0 < eights) put(c0, kept[0]);
                        if (c0 + step < eights) put(c0 + step, kept[1]);
                        for (int c = c0 + 2 * step; c < eights; c += step) put(c, get(c));
                    }
                } else {
                    if (tid < tokens) s.sx[tid] = __ldcg(a.sx + row0 + t0 + tid);
                    for (int i = tid; i < tokens * steps * 8; i += kThreads) {
                        const int t = i / (steps * 8), c = i % (steps * 8);
                        const int64_t r = row0 + t0 + t;
                        const uint4 h = __ldcg(reinterpret_cast<const uint4*>(a.x + ((int64_t)(k0 + c / 8) * a.room + r) * 64 + ((c % 8) ^ (int)(r % 8)) * 8));
                        *reinterpret_cast<uint2*>(&s.x[t][8 * c]) = make_uint2(bytes_of(make_uint2(h.x, h.y)), bytes_of(make_uint2(h.z, h.w)));
                    }
                }
                __syncthreads();
                while (now.g < groups) {
                    At then = now;
                    advance(then, kWarps, p.per);
                    if (then.g < groups) load(p, then, next);
                    if (tokens == 1) dot<1>(s, now, w);
                    else if (tokens == 2) dot<2>(s, now, w);
                    else dot<4>(s, now, w);
                    now = then;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r) w[u][r] = next[u][r];
                }
                __syncthreads();
            }
            const int rows = (int)(n1 - n0);
            for (int i = tid; i < (GATED ? rows / 2 : rows) * tokens; i += kThreads) {
                const int t = i % tokens, r = i / tokens * (GATED ? 2 : 1);
                const float* sw = a.sw + (int64_t)e * a.N + n0 + r;
                float v = (float)s.acc[t][r] * s.sx[t] * __ldg(sw);
                if (GATED) v = int8_gated(v, (float)s.acc[t][r + 1] * s.sx[t] * __ldg(sw + 1));
                const int64_t to = (first + t0 + t) * a.ldy + (n0 + r) / (GATED ? 2 : 1);
                if (y_dtype == MOE_F32) store<float>(a.y, to, v);
                else if (y_dtype == MOE_BF16) store<__nv_bfloat16>(a.y, to, v);
                else store<__half>(a.y, to, v);
            }
            __syncthreads();
            for (int i = tid; i < kRows * kTokens; i += kThreads) (&s.acc[0][0])[i] = 0;
            __syncthreads();
        }
    }
    if (!waited) pdl_wait();
}

template <typename X>
cudaError_t launch(const Int8ProductArgs& a, moe_dtype dtype, bool gated, const void* x, int64_t ldx, const int32_t* inv, int k, cudaStream_t st) {
    const X* from = static_cast<const X*>(x);
    int y_dtype = dtype;
    void* args[] = {const_cast<Int8ProductArgs*>(&a), &from, &ldx, &inv, &k, &y_dtype};
    return launch_kernel(gated ? (const void*)int8_dot_kernel<X, true> : (const void*)int8_dot_kernel<X, false>, dim3(sm_count()), dim3(kThreads),
                         sizeof(Shared), st, true, args);
}

}  // namespace

cudaError_t launch_int8_dot(const Int8ProductArgs& a, moe_dtype dtype, bool gated, const void* x, moe_dtype x_dtype, int64_t ldx,
                            const int32_t* inv, int k, cudaStream_t st) {
    if (!x) return launch<void>(a, dtype, gated, x, ldx, inv, k, st);
    switch (x_dtype) {
        case MOE_F32: return launch<float>(a, dtype, gated, x, ldx, inv, k, st);
        case MOE_BF16: return launch<__nv_bfloat16>(a, dtype, gated, x, ldx, inv, k, st);
        default: return launch<__half>(a, dtype, gated, x, ldx, inv, k, st);
    }
}

}  // namespace moe
