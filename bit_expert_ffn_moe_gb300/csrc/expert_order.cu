// expert_order.cu -- the order of (token, slot) pairs by expert: a stable counting sort of the pairs p = t k + j by ids[p].
//   offsets[e] = pairs of the experts before e;  inv[p] = offsets[ids[p]] + pairs before p with the same id, -1 without an expert
// One launch of one CTA, or of a cluster of eight for more than kOneCta pairs.  A CTA takes an equal share of the pairs, a warp
// of it an equal share of those; every warp counts its pairs per expert in shared memory, the counts are added up over
// warps and (through distributed shared memory) over CTAs, and then every warp walks its pairs once more, 32 at a time: lanes
// with the same id find each other by a ballot for each bit of the ids (a match instruction: 22 us instead of 17 for 131072
// pairs of 256 experts), and the warp's own running place of that expert moves on.  So the order does not
// depend on the order of atomics.  Bound by its chain of dependent steps: 32768 pairs of 128 experts read and write 264 KB in 6.8 us.
#include "ops.cuh"

namespace moe {
namespace {

constexpr int kOneCta = 1024;  // pairs that one CTA sorts sooner than a cluster
constexpr int kClusterCtas = 8;
constexpr int kKept = 8;  // turns of 32 ids that a warp keeps in registers from its first walk for its second

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
    auto id_at = [&](int p) {
        const int e = p < p1 ? __ldg(ids + p) : -1;
        return (unsigned)e < (unsigned)E ? e : -1;
    };
    int kept[kKept];
#pragma unroll
    for (int i = 0; i < kKept; ++i) kept[i] = id_at(p0 + 32 * i + lane);
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        if (kept[i] >= 0) atomicAdd(&mine[kept[i]], 1);
    for (int p = p0 + 32 * kKept + lane; p < p1; p += 32) {
        const int e = id_at(p);
        if (e >= 0) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    // `group` neighbouring threads add up an expert's counts, each those of a few consecutive warps
    int group = 1;
    while (group < 8 && 2 * group * E <= (int)blockDim.x && warps % (2 * group) == 0) group *= 2;
    for (int i = threadIdx.x; i / group < (E + 31) / 32 * 32; i += blockDim.x) {  // (whole warps)
        const int e = i / group, part = i % group, each = warps / group;
        int sum = 0, incl;
        if (e < E)
            for (int w = part * each; w < (part + 1) * each; ++w) sum += counts[w * E + e];
        incl = sum;
        for (int o = 1; o < group; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (part >= o) incl += v;
        }
        if (e >= E) continue;
        int run = incl - sum;
        for (int w = part * each; w < (part + 1) * each; ++w) {
            const int c = counts[w * E + e];
            counts[w * E + e] = run;
            run += c;
        }
        if (part == group - 1) total[e] = run;
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
            int n[kClusterCtas];
#pragma unroll
            for (int c = 0; c < kClusterCtas; ++c) n[c] = ld_peer(total + e, c);
#pragma unroll
            for (int c = 0; c < kClusterCtas; ++c) {
                before += c < (int)blockIdx.x ? n[c] : 0;
                all += n[c];
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
    const int bits = 33 - __clz(E);  // (-1 has all of them set, no id the last one)
    auto walk = [&](int p, int e) {
        unsigned same = 0xffffffffu;
        for (int b = 0; b < bits; ++b) {
            const unsigned set = __ballot_sync(0xffffffffu, (e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        const int before = __popc(same & ((1u << lane) - 1u));
        const int r = e >= 0 ? place[e] + mine[e] + before : -1;
        __syncwarp();
        if (e >= 0 && before == 0) mine[e] += __popc(same);
        __syncwarp();
        if (p < p1) inv[p] = r;
    };
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        if (p0 + 32 * i < p1) walk(p0 + 32 * i + lane, kept[i]);
    for (int q = p0 + 32 * kKept; q < p1; q += 32) walk(q + lane, id_at(q + lane));
    if (ctas > 1) cluster_wait();  // no CTA's totals go before all have read them
}

}  // namespace

cudaError_t launch_expert_order(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* inv, cudaStream_t st) {
    int ctas = P > kOneCta ? kClusterCtas : 1;
    // A warp for every 64 pairs or so, and room for their counts.  More than 16 only where these could not keep their pairs (us for 32768
    // pairs of 128 experts with 8, 16, 32 warps: 9.8, 6.8, 8.5; for 131072 of 256: 34, 21, 17).
    int warps = (P / ctas + 63) / 64;
    warps = warps < 4 ? 4 : warps <= 16 ? warps : P / ctas <= 16 * 32 * kKept ? 16 : 32;
    const size_t smem = sizeof(int) * (size_t)(warps + 2) * E;
    const void* f = (const void*)expert_order_kernel;
    cudaError_t e = ensure_dyn_smem(f, smem);
    if (e != cudaSuccess) return e;
    void* args[] = {&ids, &P, &E, &ctas, &offsets, &inv};
    return launch_cluster(f, dim3(ctas), warps * 32, smem, ctas, st, args);
}

}  // namespace moe
