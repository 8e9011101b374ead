// int8_few.cu -- the 8-bit products of a few dozen rows with one matrix, on the tensor cores: a tile of 128 weight rows by all rows (or
// up to 128 of them) for a cluster of CTAs that share its K range; their sums are exchanged through distributed shared memory
// and added in rank order, each CTA storing its share of the rows.  Bound by the weight read: every CTA's first copies
// start before anything else, and there is one tile a CTA, so that nothing has to be found out about the work first.
//   warps 0-15  conversion of the weights (int8_mma.cu), then results out of tensor memory
//   warp 16     copies            warp 17     products
// 16 x 4096 x 8192 (33.6 MB): 11.7 us, 777 x 1001 x 1543: 9.0.
// Every barrier wait is bounded: on expiry the CTA records MOE_ERR_TIMEOUT, waits (bounded) for its own copies and products,
// frees tensor memory and exits.
#include "int8_mma.cuh"

namespace moe {
namespace {

constexpr int kSets = 4, kConvWarps = 4 * kSets, kCopyWarp = kConvWarps, kMmaWarp = kCopyWarp + 1;
constexpr int kWarps = kMmaWarp + 1, kThreads = 32 * kWarps;
constexpr int kMostRows = 128, kMostStages = 10;
constexpr uint32_t kTmemCols = 256, kSlotCols = 32, kSlotBase = kMostRows;
static_assert(kSlotBase + kSets * kSlotCols == kTmemCols, "tensor memory");

struct Shared {
    uint64_t full[kMostStages], ready[kMostStages], empty[kMostStages], done;
    uint32_t tmem;
    volatile int abort;
};
struct FewArgs {
    Int8ProductArgs p;
    int y_dtype, splits, n, stages, x_bytes, stage_bytes;  // CTAs of a tile; its rows; the ring; its rows' bytes of a tile of weights
};

// Four floats at the place of p in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_peer4(const float* p, int rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(smem_u32(p)), "r"(rank)
        : "memory");
    return v;
}

template <typename T, bool GATED>
__device__ __forceinline__ void store4(void* y, int64_t row, int n, int N, const float (&v)[4], bool wide) {
    T* to = static_cast<T*>(y) + row + (GATED ? n / 2 : n);
    if constexpr (GATED) {
        const T u[2] = {int8_result<T>(int8_gated(v[0], v[1])), int8_result<T>(int8_gated(v[2], v[3]))};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (n + 2 * i < N) to[i] = u[i];
    } else {
        __align__(16) T u[4] = {int8_result<T>(v[0]), int8_result<T>(v[1]), int8_result<T>(v[2]), int8_result<T>(v[3])};
        if (wide && n + 4 <= N) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(u);
            else *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(u);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < N) to[i] = u[i];
        }
    }
}

// Grid: x = weight tile * splits + rank, y = activation tile.
template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1) int8_few_kernel(const __grid_constant__ FewArgs args) {
    const Int8ProductArgs& a = args.p;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared& s = *reinterpret_cast<Shared*>(ring + (size_t)args.stages * args.stage_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = args.stages, splits = args.splits;
    const int rank = (int)blockIdx.x % splits, nt = (int)blockIdx.x / splits, m0 = (int)blockIdx.y * args.n;
    const int KT = (int)((a.K + 63) / 64), KS = (KT + 1) / 2, k0 = KS * rank / splits, steps = KS * (rank + 1) / splits - k0;
    const int live = min(args.n, (int)a.M - m0);
    int* const status = &a.ctrl->status;

    if (warp == kCopyWarp) {
        if (lane < S) {
            mbar_init(&s.full[lane], 1);
            mbar_init(&s.ready[lane], 8);
            mbar_init(&s.empty[lane], 1);
        }
        if (lane == 0) mbar_init(&s.done, 1), s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
    }
    const uint32_t full0 = smem_u32(s.full), ring0 = smem_u32(ring);
    const uint8_t* w = a.w + ((int64_t)nt * KT + 2 * k0) * kInt8Tile;
    const int head = min(S, steps), bytes = min(args.n, (live + 15) / 16 * 16) * 128;
    if (warp == kCopyWarp && elect_one()) {  // the first weights at once, if they may
        if (!a.early) pdl_wait();
        for (int i = 0; i < head; ++i, w += 2 * kInt8Tile) {
            const int tiles = min(2, KT - 2 * (k0 + i));
            expect_bytes(full0 + 8 * i, tiles * (kInt8Tile + bytes));
            bulk_copy(ring0 + i * args.stage_bytes + 2 * args.x_bytes, w, tiles * kInt8Tile, full0 + 8 * i);
        }
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;

    if (warp == kCopyWarp) {
        if (elect_one()) {
            pdl_wait();
            const int64_t x_step = a.room * 128;
            const uint8_t* x = reinterpret_cast<const uint8_t*>(a.x) + 2 * k0 * x_step + (int64_t)m0 * 128;
            Turn t(S);
            w = a.w + ((int64_t)nt * KT + 2 * (k0 + head)) * kInt8Tile;
            int it = 0;
            for (; it < steps; ++it, x += 2 * x_step, t.next()) {
                const uint32_t bar = full0 + 8 * t.at, to = ring0 + t.at * args.stage_bytes;
                const int tiles = min(2, KT - 2 * (k0 + it));
                if (it >= head) {
                    if (!mbar_wait(&s.empty[t.at], t.parity ^ 1, &s.abort, status)) break;
                    expect_bytes(bar, tiles * (kInt8Tile + bytes));
                    bulk_copy(to + 2 * args.x_bytes, w, tiles * kInt8Tile, bar);
                    w += 2 * kInt8Tile;
                }
                bulk_copy(to, x, bytes, bar);
                if (tiles == 2) bulk_copy(to + args.x_bytes, x + x_step, bytes, bar);
            }
            land(s.full, it, S);
        }
    } else if (warp == kMmaWarp) {
        if (elect_one()) {
            const uint32_t idesc = idesc_f16(128, args.n);
            uint32_t slot = tmem + kSlotBase;
            Turn t(S);
            for (int k = 0; k < steps; ++k, t.next(), slot ^= 2 * kSlotCols) {
                if (!mbar_wait(&s.ready[t.at], t.parity, &s.abort, status)) break;
                tc_fence_after();
                const uint32_t x = ((ring0 + t.at * args.stage_bytes) >> 4) | (1u << 16);
                step_products<false>(tmem, slot, x, idesc, k > 0 ? 1u : 0u);
                if (2 * (k0 + k) + 1 < KT) step_products<false>(tmem, slot + kSlotCols, x + (args.x_bytes >> 4), idesc, 1u);
                commit<false>(&s.empty[t.at]);
            }
            commit<false>(&s.done);
        }
    } else {
        const int set = warp >> 2, q = warp & 3;
        const unsigned char* w0 = ring + 2 * args.x_bytes + (set & 1) * kInt8Tile + (32 * q + lane) * 16;
        const uint32_t slot = tmem + ((uint32_t)(32 * q) << 16) + kSlotBase + set * kSlotCols;
        Turn t(S), old(S);  // the step; the one before the last
        for (int k = 0; k < steps; ++k, t.next()) {
            if (k >= 3) old.next();
            if ((k & 1) != set >> 1) continue;
            // (Of the set's own steps alone: the copies of another's can be followed by the next ones in their place before this set looks.  Own
            // phases are not mistaken: the step that had the place before, S >= 4 steps ago, had been multiplied when this set's
            // last step took its slot; and the step that has it next waits for this one's products.)
            if (!mbar_wait_warp(&s.full[t.at], t.parity, &s.abort, status)) break;
            if (2 * (k0 + k) + (set & 1) < KT) {
                uint32_t h[32];
                convert_row(w0 + (size_t)t.at * args.stage_bytes, h);
                // the products of the step before the last have read this slot (its phase is not mistaken: this step was copied
                // after the products of the step S before had completed)
                if (k >= 2 && !mbar_wait_warp(&s.empty[old.at], old.parity, &s.abort, status)) break;
                tc_fence_after();
                tmem_st32(slot, h);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.ready[t.at]);
        }
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
    // This lane's four weight rows, and this warp's activation rows: their scales are on their way while the last products run
    const int n = nt * 128 + 4 * lane, N = (int)a.N;
    float sw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sw[i] = n + i < N ? __ldg(a.sw + n + i) : 0.f;
    int c = rank + splits * warp;
    float sx = c < live ? __ldcg(a.sx + m0 + c) : 0.f;
    {
        // every product has completed: the commit comes, aborting or not
        volatile int never = 0;
        mbar_wait(&s.done, 0, &never, status);
    }
    tc_fence_after();
    __syncthreads();  // and no copy is in flight: they have landed, or (bounded) been waited for

    // Results go through shared memory, [activation row][128 weight rows], on the ring.
    float* part = reinterpret_cast<float*>(ring);
    if (warp < kConvWarps) {
        const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        for (int c0 = 16 * (warp >> 2); c0 < live; c0 += 16 * kSets) {
            uint32_t v[16];
            tmem_ld16(acc + c0, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c0 + i) * 128 + 32 * (warp & 3) + lane] = __uint_as_float(v[i]);
        }
    }
    tc_fence_before();
    if (splits > 1) {
        __syncwarp();
        cluster_sync();
    } else {
        __syncthreads();
    }
    const int64_t size = args.y_dtype == MOE_F32 ? 4 : 2;
    const bool wide = reinterpret_cast<uintptr_t>(a.y) % (4 * size) == 0 && a.ldy % 4 == 0;
    while (c < live) {
        const float* from = part + c * 128 + 4 * lane;
        float4 o[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < splits) o[r] = splits > 1 ? ld_peer4(from, r) : *reinterpret_cast<const float4*>(from);
        float4 sum = o[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
            if (r < splits) sum.x += o[r].x, sum.y += o[r].y, sum.z += o[r].z, sum.w += o[r].w;
        const float v[4] = {sum.x * sx * sw[0], sum.y * sx * sw[1], sum.z * sx * sw[2], sum.w * sx * sw[3]};
        const int64_t row = (int64_t)(m0 + c) * a.ldy;
        if (n < N) {
            if (args.y_dtype == MOE_F32) store4<float, GATED>(a.y, row, n, N, v, wide);
            else if (args.y_dtype == MOE_BF16) store4<__nv_bfloat16, GATED>(a.y, row, n, N, v, wide);
            else store4<__half, GATED>(a.y, row, n, N, v, wide);
        }
        c += splits * kWarps;
        if (c < live) sx = __ldcg(a.sx + m0 + c);
    }
    if (splits > 1) {
        __syncwarp();
        cluster_sync();  // the partial sums stay until every CTA has read them
    } else {
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

}  // namespace

bool int8_few_fits(const Int8ProductArgs& a) {
    const int64_t tiles = ((a.N + 127) / 128) * ((a.M + kMostRows - 1) / kMostRows);
    return !a.offsets && tiles <= sm_count();
}

cudaError_t launch_int8_few(const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st) {
    FewArgs f = {};
    f.p = a;
    f.y_dtype = dtype;
    const int nt = (int)((a.N + 127) / 128), mt = (int)((a.M + kMostRows - 1) / kMostRows), KS = (int)((a.K + 127) / 128);
    f.n = ((int)((a.M + mt - 1) / mt) + 15) / 16 * 16;
    // CTAs that share a tile's K range: as many as leave every one its own SM and at least two steps
    f.splits = 1;
    while (f.splits < 8 && nt * mt * f.splits * 2 <= sm_count() && KS / (f.splits * 2) >= 2) f.splits *= 2;
    f.x_bytes = (f.n * 128 + 1023) / 1024 * 1024;
    f.stage_bytes = 2 * (f.x_bytes + kInt8Tile);
    const int fit = (int)((232448 - 1024 - sizeof(Shared)) / f.stage_bytes);
    f.stages = fit < kMostStages ? fit : kMostStages;  // (4 at least)
    // (more than half of the SM's shared memory, so that CTAs do not share its tensor memory)
    size_t smem = (size_t)f.stages * f.stage_bytes + sizeof(Shared) + 1024;
    if (smem < 120 * 1024) smem = 120 * 1024;
    void* args[] = {&f};
    return launch_cluster(gated ? (const void*)int8_few_kernel<true> : (const void*)int8_few_kernel<false>, dim3(nt * f.splits, mt), kThreads, smem,
                          f.splits, st, args);
}

}  // namespace moe
