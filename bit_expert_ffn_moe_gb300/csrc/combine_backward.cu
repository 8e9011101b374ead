// combine_backward.cu -- gradients of the weighted sum y[t] = sum_j w[t][j] y_perm[inv_pos[t k + j]]:
//   dw[t][j] = <dy[t], y_perm[inv_pos[t k + j]]>   (fp32 sums)
//   dy_perm[inv_pos[t k + j]] = w[t][j] dy[t]      (rounded once to bf16)
// The k rows of a token are read and written once; dy[t] is read once per eight slots (the first time
// from memory).  Bound by HBM: 2 T d + 4 T k d bytes; 4096 tokens x 8 slots x 8192 features: 180 us, 6.35 TB/s (two CTAs per SM
// instead of three: 185).
#include "ops.cuh"
#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kMostThreads = 320;

// `warps` warps of a CTA share a token: thread c of them the 8-feature pieces c, c + 32 warps, ...  SLOTS slots of a token are
// in registers at a time, and PIECES pieces of each, so that tokens of few slots have as many loads in flight (6546 tokens of
// one slot, d = 6632: 46.8 us, 81 with one piece; 800 tokens of 12 slots, d = 6448: 46.8 us as 6 + 6, 54 as 8 + 4).
template <int SLOTS, int PIECES>
__global__ void __launch_bounds__(kMostThreads, 3)
    combine_backward_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ y_perm,
                            const int32_t* __restrict__ inv_pos, const float* __restrict__ w, int T, int k, int d, int warps,
                            float* __restrict__ dw, uint16_t* __restrict__ dy_perm) {
    __shared__ float part[kMostThreads / 32][SLOTS];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tokens = (int)(blockDim.x >> 5) / warps, mine = warp / warps;  // tokens per CTA, this warp's token
    const int64_t t = (int64_t)blockIdx.x * tokens + mine;
    const bool live = t < T;
    const int first = threadIdx.x - mine * warps * 32, step = warps * 32, pieces = d / 8;
    for (int j0 = 0; j0 < k; j0 += SLOTS) {
        int64_t r[SLOTS];
        float wj[SLOTS], acc[SLOTS];
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const int p = live && j0 + q < k ? __ldg(inv_pos + t * k + j0 + q) : -1;
            r[q] = (unsigned)p < (unsigned)(T * k) ? p : -1;  // else not a row of y_perm: takes no part
            wj[q] = r[q] >= 0 && w ? __ldg(w + t * k + j0 + q) : 0.f;
            acc[q] = 0.f;
        }
        if (live)
            for (int c0 = first; c0 < pieces; c0 += PIECES * step) {
                uint4 g[PIECES], y[PIECES][SLOTS];
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    const int c = c0 + i * step;
                    const bool in = PIECES == 1 || c < pieces;
                    g[i] = in ? *reinterpret_cast<const uint4*>(dy + t * d + 8 * c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int q = 0; q < SLOTS; ++q)
                        y[i][q] = in && dw && r[q] >= 0 ? __ldcs(reinterpret_cast<const uint4*>(y_perm + r[q] * d + 8 * c))
                                                        : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    const int c = c0 + i * step;
                    if (PIECES > 1 && c >= pieces) break;
                    const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
                    for (int q = 0; q < SLOTS; ++q) {
                        if (r[q] < 0) continue;
                        const uint32_t yw[4] = {y[i][q].x, y[i][q].y, y[i][q].z, y[i][q].w};
                        uint32_t o[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const float lo = bf16_bits_to_f32(gw[m] & 0xFFFF), hi = bf16_bits_to_f32(gw[m] >> 16);
                            acc[q] = fmaf(lo, bf16_bits_to_f32(yw[m] & 0xFFFF), acc[q]);
                            acc[q] = fmaf(hi, bf16_bits_to_f32(yw[m] >> 16), acc[q]);
                            o[m] = (uint32_t)f32_to_bf16_bits(wj[q] * lo) | ((uint32_t)f32_to_bf16_bits(wj[q] * hi) << 16);
                        }
                        if (dy_perm)
                            __stcs(reinterpret_cast<uint4*>(dy_perm + r[q] * d + 8 * c), make_uint4(o[0], o[1], o[2], o[3]));
                    }
                }
            }
        if (!dw) continue;
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            acc[q] = warp_butterfly_sum(acc[q]);
            if (lane == 0) part[warp][q] = acc[q];
        }
        __syncthreads();
        if (live && warp % warps == 0 && lane < SLOTS && j0 + lane < k) {
            float sum = 0.f;
            for (int v = 0; v < warps; ++v) sum += part[warp + v][lane];
            dw[t * k + j0 + lane] = sum;
        }
        __syncthreads();
    }
}

struct Variant {
    const void* kernel;
    int pieces;
};
template <int SLOTS, int PIECES>
Variant variant_of() {
    return {(const void*)combine_backward_kernel<SLOTS, PIECES>, PIECES};
}
Variant variant(int slots) {
    switch (slots) {
        case 1: return variant_of<1, 4>();
        case 2: return variant_of<2, 2>();
        case 3: return variant_of<3, 2>();
        case 4: return variant_of<4, 2>();
        case 5: return variant_of<5, 1>();
        case 6: return variant_of<6, 1>();
        case 7: return variant_of<7, 1>();
        default: return variant_of<8, 1>();
    }
}

}  // namespace

cudaError_t launch_combine_backward(const uint16_t* dy, const uint16_t* y_perm, const int32_t* inv_pos, const float* w,
                                    int T, int k, int d, float* dw, uint16_t* dy_perm, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    // slots in turns of up to eight, as even as they go
    const int turns = (k + 7) / 8, slots = (k + turns - 1) / turns;
    const Variant v = variant(slots);
    // enough threads for one or more turns each: 1, 2 or 4 warps a token and several tokens a CTA, or one token and as
    // many warps as hold it (2056 features, 333 tokens: 7.4 us with 8 warps, whose second turn had one thread at work)
    const int pieces = (d / 8 + v.pieces - 1) / v.pieces;
    int threads = kThreads, warps = 1;
    while (warps < kThreads / 32 && warps * 32 < pieces) warps *= 2;
    if (pieces > kThreads && pieces <= kMostThreads) threads = kMostThreads, warps = kMostThreads / 32;
    const int tokens = threads / 32 / warps;
    void* args[] = {&dy, &y_perm, &inv_pos, &w, &T, &k, &d, &warps, &dw, &dy_perm};
    return launch_kernel(v.kernel, dim3((T + tokens - 1) / tokens), dim3(threads), 0, st, true,
                         args);
}

}  // namespace moe
