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
constexpr int kSlots = 8;  // slots of a token in registers at a time

// `warps` warps of a CTA share a token: thread c of them the 8-feature pieces c, c + 32 warps, ...
__global__ void __launch_bounds__(kMostThreads, 3)
    combine_backward_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ y_perm,
                            const int32_t* __restrict__ inv_pos, const float* __restrict__ w, int T, int k, int d, int warps,
                            float* __restrict__ dw, uint16_t* __restrict__ dy_perm) {
    __shared__ float part[kMostThreads / 32][kSlots];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tokens = (int)(blockDim.x >> 5) / warps, mine = warp / warps;  // tokens per CTA, this warp's token
    const int64_t t = (int64_t)blockIdx.x * tokens + mine;
    const bool live = t < T;
    const int first = threadIdx.x - mine * warps * 32, step = warps * 32, pieces = d / 8;
    for (int j0 = 0; j0 < k; j0 += kSlots) {
        int64_t r[kSlots];
        float wj[kSlots], acc[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            const int p = live && j0 + q < k ? __ldg(inv_pos + t * k + j0 + q) : -1;
            r[q] = (unsigned)p < (unsigned)(T * k) ? p : -1;  // else not a row of y_perm: takes no part
            wj[q] = r[q] >= 0 && w ? __ldg(w + t * k + j0 + q) : 0.f;
            acc[q] = 0.f;
        }
        if (live)
            for (int c = first; c < pieces; c += step) {
                const uint4 g = *reinterpret_cast<const uint4*>(dy + t * d + 8 * c);
                const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
                uint4 y[kSlots];
#pragma unroll
                for (int q = 0; q < kSlots; ++q)
                    y[q] = dw && r[q] >= 0 ? __ldcs(reinterpret_cast<const uint4*>(y_perm + r[q] * d + 8 * c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < kSlots; ++q) {
                    if (r[q] < 0) continue;
                    const uint32_t yw[4] = {y[q].x, y[q].y, y[q].z, y[q].w};
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
        if (!dw) continue;
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            acc[q] = warp_butterfly_sum(acc[q]);
            if (lane == 0) part[warp][q] = acc[q];
        }
        __syncthreads();
        if (live && warp % warps == 0 && lane < kSlots && j0 + lane < k) {
            float sum = 0.f;
            for (int v = 0; v < warps; ++v) sum += part[warp + v][lane];
            dw[t * k + j0 + lane] = sum;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_combine_backward(const uint16_t* dy, const uint16_t* y_perm, const int32_t* inv_pos, const float* w,
                                    int T, int k, int d, float* dw, uint16_t* dy_perm, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    // enough threads for one or more pieces each: 1, 2 or 4 warps a token and several tokens a CTA, or one token and as
    // many warps as hold it (2056 features, 333 tokens: 7.4 us with 8 warps, whose second turn had one thread at work)
    const int pieces = d / 8;
    int threads = kThreads, warps = 1;
    while (warps < kThreads / 32 && warps * 32 < pieces) warps *= 2;
    if (pieces > kThreads && pieces <= kMostThreads) threads = kMostThreads, warps = kMostThreads / 32;
    const int tokens = threads / 32 / warps;
    void* args[] = {&dy, &y_perm, &inv_pos, &w, &T, &k, &d, &warps, &dw, &dy_perm};
    return launch_kernel((const void*)combine_backward_kernel, dim3((T + tokens - 1) / tokens), dim3(threads), 0, st, true,
                         args);
}

}  // namespace moe
