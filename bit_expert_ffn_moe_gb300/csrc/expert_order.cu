// expert_order.cu -- the order of (token, slot) pairs by expert: a stable counting sort of the pairs p = t k + j by ids[p].
//   offsets[e] = pairs of the experts before e;  inv[p] = offsets[ids[p]] + pairs before p with the same id, -1 without an expert
// One launch of one CTA, or of a cluster of eight for more than kOneCta pairs.  A CTA takes an equal share of the pairs, a warp
// of it an equal share of those; every warp counts its pairs per expert in shared memory, the counts are added up over
// warps and (through distributed shared memory) over CTAs, and then every warp walks its pairs once more, 32 at a time: lanes
// with the same id find each other by match_any, and the warp's own running place of that expert moves on.  So the order does not
// depend on the order of atomics.  Bound by its chain of dependent steps; 32768 pairs of 128 experts read and write 264 KB.
#include "ops.cuh"

namespace moe {
namespace {

constexpr int kOneCta = 2048;  // pairs that one CTA sorts sooner than a cluster
constexpr int kClusterCtas = 8;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The int at the place of p in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ int ld_peer(const int* p, int rank) {
    int v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %1, %2;\n\t"
        "ld.shared::cluster.s32 %0, [a];\n\t}"
        : "=r"(v)
        : "r"(smem_u32(p)), "r"(rank)
        : "memory");
    return v;
}

// Shared memory: counts [warps][E], then the CTA's own totals [E], then the first place [E] of its pairs.
__global__ void __launch_bounds__(1024)
    expert_order_kernel(const int32_t* __restrict__ ids, int P, int E, int ctas, int32_t* __restrict__ offsets, int32_t* __restrict__ inv) {
    extern __shared__ int counts[];
    __shared__ int scan[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int* total = counts + warps * E;
    int* place = total + E;
    int* mine = counts + warp * E;
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x) counts[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    // (64-bit products: P up to 2^30 times the number of warps)
    const int64_t share = blockIdx.x * warps + warp, shares = (int64_t)ctas * warps;
    const int p0 = (int)(P * share / shares), p1 = (int)(P * (share + 1) / shares);
    for (int p = p0 + lane; p < p1; p += 32) {
        const int e = ids[p];
        if ((unsigned)e < (unsigned)E) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int run = 0;
        for (int w = 0; w < warps; ++w) {
            const int c = counts[w * E + e];
            counts[w * E + e] = run;
            run += c;
        }
        total[e] = run;
    }
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // thread i: experts i per, ... (consecutive ones); exclusive sums over all of them
    const int per = (E + blockDim.x - 1) / blockDim.x, e0 = min(E, (int)threadIdx.x * per), e1 = min(E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int all = 0, before = 0;
        if (ctas == 1) {
            all = total[e];
        } else {
            for (int c = 0; c < ctas; ++c) {
                const int n = ld_peer(total + e, c);
                before += c < (int)blockIdx.x ? n : 0;
                all += n;
            }
        }
        place[e] = sum + before;
        if (blockIdx.x == 0) offsets[e] = sum;
        sum += all;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int v = lane < warps ? scan[lane] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        scan[lane] = s - v;
        if (blockIdx.x == 0 && lane == 31) offsets[E] = s;
    }
    if (ctas > 1) cluster_arrive();  // (the totals have been read)
    __syncthreads();
    const int base = scan[warp] + incl - sum;
    for (int e = e0; e < e1; ++e) {
        place[e] += base;
        if (blockIdx.x == 0 && base) offsets[e] += base;
    }
    __syncthreads();
    for (int q = p0; q < p1; q += 32) {
        const int p = q + lane;
        int e = p < p1 ? ids[p] : -1;
        if ((unsigned)e >= (unsigned)E) e = -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int r = e >= 0 ? place[e] + mine[e] + before : -1;
        __syncwarp();
        if (e >= 0 && before == 0) mine[e] += __popc(same);
        __syncwarp();
        if (p < p1) inv[p] = r;
    }
    if (ctas > 1) cluster_wait();  // no CTA's totals go before all have read them
}

}  // namespace

cudaError_t launch_expert_order(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* inv, cudaStream_t st) {
    int ctas = P > kOneCta ? kClusterCtas : 1;
    // a warp for every 32 pairs or so, and room for their counts
    int warps = (P / ctas + 31) / 32;
    warps = warps < 4 ? 4 : warps > 32 ? 32 : warps;
    const size_t smem = sizeof(int) * (size_t)(warps + 2) * E;
    const void* f = (const void*)expert_order_kernel;
    cudaError_t e = ensure_dyn_smem(f, smem);
    if (e != cudaSuccess) return e;
    void* args[] = {&ids, &P, &E, &ctas, &offsets, &inv};
    return launch_cluster(f, dim3(ctas), warps * 32, smem, ctas, st, args);
}

}  // namespace moe
