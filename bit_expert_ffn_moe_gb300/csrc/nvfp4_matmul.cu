// nvfp4_matmul.cu -- dense product of two NVFP4 operands on the tensor cores (kind::mxf4nvf4):
//   y[m][n] = ga[m] gb[n] sum_k A[m][k] B[n][k],
// A [M][K] the activations, B [N][K] the weights (or any two operands that contract along K), both in
// the tensor-core layout of nvfp4_operand.cu: code tiles of 128 rows x 256 values with the 128-byte swizzle and
// 512-byte scale atoms, so that every piece is one contiguous bulk copy and ragged sizes need no
// masks before the store (padding along K holds zeros; padding rows only reach results that are not stored).
// Products and sums are the tensor core's (fp32 accumulators); each result is multiplied by ga, then by gb, in fp32
// and rounded to y's type.
//
// Two kernels:
//   rows    up to 128 activation rows per tile: the weights are the MMA's M side (128 weight rows), the
//           activations its N side (8 .. 128 rows), so that few activation rows waste no tensor-core rows
//           and each weight byte is read once.  Bound by the weight read; the K range of a tile is split
//           over the CTAs of a cluster, whose partial sums are exchanged through distributed shared
//           memory and added in rank order.
//           16 x 4096 x 8192: 6 us with its launch, 3.2 TB/s; 4 us of it are the kernel's fixed chain (set-up, first
//           copies, last products, exchange, store).
//   pair    more rows: 256 x 256 tiles by pairs of CTAs, persistent.  8192^3: 152 us, 7.2 PFLOP/s; 4096 x 4096 x 8192: 45.6 us
//           (256 tiles in 4 waves of 76 pairs).  A K step takes 540 cycles, of which 300 are what it takes to write its
//           operands to shared memory and 250 .. 380 to read them; a tile adds about 600 cycles without products while
//           its results are read.
// Every barrier wait is bounded: on expiry the CTA records MOE_ERR_TIMEOUT, waits (bounded) for its own
// copies and MMAs, frees tensor memory and exits.
#include "ops.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kTile = 128 * 128;  // code tile: 128 rows x 128 bytes (256 values)
constexpr int kAtom = 512;        // scale atom: 128 rows x 4 scales
constexpr int kAtoms = 4;         // scale atoms of 128 rows per K step of 256 values
constexpr uint32_t kTmemCols = 512;

struct MatmulArgs {
    const uint8_t* qa;
    const uint8_t* sa;
    const float* ga;
    int ga_rows;
    const uint8_t* qb;
    const uint8_t* sb;
    const float* gb;
    int gb_rows;
    int64_t M, N;
    int KT;  // K steps of 256 values
    void* y;
    int dtype;
    int64_t ldy;
    int* status;
    int weights_ready;  // B is there before the kernel before has ended
};

template <typename T>
__device__ __forceinline__ T out_value(float v);
template <>
__device__ __forceinline__ float out_value<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 out_value<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half out_value<__half>(float v) { return __float2half_rn(v); }

// 16 bytes of results from consecutive fp32 values.
template <typename T>
__device__ __forceinline__ uint4 out_piece(const uint32_t* v) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            o[i] = v[i];
        } else {
            const T lo = out_value<T>(__uint_as_float(v[2 * i])), hi = out_value<T>(__uint_as_float(v[2 * i + 1]));
            o[i] = (uint32_t)*reinterpret_cast<const uint16_t*>(&lo) | ((uint32_t)*reinterpret_cast<const uint16_t*>(&hi) << 16);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A result is (sum * ga) * gb.  Its first product leaves fp32's range only where a row's scale is far from 1 (a sum is 0 or 2^-20 ..
// 2^45; a row of the type's largest numbers has a scale of 2^117): then all rows' scales of the warp times a power of two and
// the columns' scales divided by it, which is exact, keep what fp32 can hold.
__device__ __forceinline__ bool far_scale(float ga) { return ga > 0x1p80f || ga < 0x1p-100f; }
// That power of two for the rows' scales ga (one per lane) and the columns' between gb_min and gb_max (per lane): no further than
// leaves every scale in range.
__device__ __noinline__ float scale_shift(float ga, float gb_min, float gb_max) {
    auto exponent = [](float v) { return (int)(__float_as_uint(v) >> 23) - 127; };
    const bool counts = ga > 0.f && ga < INFINITY;
    const int a1 = __reduce_max_sync(0xffffffffu, counts ? exponent(ga) : -200), a0 = __reduce_min_sync(0xffffffffu, counts ? exponent(ga) : 200);
    const int c1 = __reduce_max_sync(0xffffffffu, exponent(gb_max)), c0 = __reduce_min_sync(0xffffffffu, exponent(gb_min));
    int p = 0;
    if (a1 > 80) p = min(max(max(80 - a1, c1 - 127), -100 - a0), 0);
    else if (a0 < -100) p = max(min(min(-100 - a0, 80 - a1), c0 + 126), 0);
    return __uint_as_float((uint32_t)(127 + p) << 23);
}

// One thread of a converged warp, known as one to the compiler: where it is chosen by its lane number instead, each copy or MMA
// is issued through a loop over the lanes (about 130 cycles; 8192^3: 165 us, 150 with this for the pair kernel's copies).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// ------------------------------------------------------------------ rows kernel
// One K step (256 values) of M = 128 weight rows x N activation rows: eight scale-atom copies, four MMAs,
// the commit that frees the stage.  Scale columns of a stage: weights' atom i at sf + 4 i, activations' at
// sf + 16 + 4 i.
__device__ __forceinline__ void rows_stage_mma(uint32_t d, uint32_t sf, uint64_t a, uint64_t b, uint64_t asf, uint64_t bsf,
                                               uint32_t idesc, uint32_t accumulate, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%2], %3;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %5;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%6], %7;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%8], %9;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%10], %11;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%12], %13;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%14], %15;\n\t}" ::"r"(sf),
        "l"(asf), "r"(sf + 4), "l"(asf + 32), "r"(sf + 8), "l"(asf + 64), "r"(sf + 12), "l"(asf + 96), "r"(sf + 16), "l"(bsf),
        "r"(sf + 20), "l"(bsf + 32), "r"(sf + 24), "l"(bsf + 64), "r"(sf + 28), "l"(bsf + 96)
        : "memory");
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 q, %4, %4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %7, %8, %3, [%9], [%10], q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %11, %12, %3, [%13], [%14], q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %15, %16, %3, [%17], [%18], q;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%19];\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sf), "r"(sf + 16), "l"(a + 2), "l"(b + 2), "r"(sf + 4), "r"(sf + 20),
        "l"(a + 4), "l"(b + 4), "r"(sf + 8), "r"(sf + 24), "l"(a + 6), "l"(b + 6), "r"(sf + 12), "r"(sf + 28),
        "r"(smem_u32(bar))
        : "memory");
}

constexpr int kRowsThreads = 192;  // copy warp, MMA warp, 4 epilogue warps

template <int NT>
__host__ __device__ constexpr int rows_stage_bytes() { return kTile + NT * 128 + 2 * kAtoms * kAtom; }
template <int NT>
__host__ __device__ constexpr int rows_stages() { return NT == 128 ? 6 : 8; }
// (more than half of the SM's shared memory, so that one CTA per SM owns its tensor memory)
template <int NT>
constexpr size_t rows_smem() { return (size_t)rows_stages<NT>() * rows_stage_bytes<NT>() + 1024 + 256; }
static_assert(rows_smem<8>() > 116 * 1024 && rows_smem<64>() <= 232448 && rows_smem<128>() <= 232448, "one CTA per SM");

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Four floats at the place of p in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_peer_f4(const void* p, uint32_t rank) {
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

// Activation rows c = rank, rank + splits, ... of a tile's results part[c][128] (summed over the cluster's CTAs in rank order),
// scaled and stored, a warp per row.  ga: the rows' scales from the tile's first row on, or one.
template <typename T, int WARPS, int NT>
__device__ __forceinline__ void store_rows(const MatmulArgs& args, const float* part, int64_t nt, int64_t m0, int rows, int rank,
                                           int splits, const float* ga, bool ga_rows) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = nt * 128 + 4 * lane;  // this lane's four weight rows
    const int live = (int)max((int64_t)0, min((int64_t)4, args.N - n));
    float gb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) gb[i] = i < live ? args.gb[args.gb_rows ? n + i : 0] : 0.f;
    const bool wide = reinterpret_cast<uintptr_t>(args.y) % 16 == 0 && args.ldy % 4 == 0;
    const int c0 = rank + splits * warp;
    float ga_lane = 1.f;  // lane i: the scale of this warp's i-th row (at most 22)
    if (c0 + splits * WARPS * lane < rows) ga_lane = ga[ga_rows ? c0 + splits * WARPS * lane : 0];
    if (__any_sync(0xffffffffu, far_scale(ga_lane))) {
        float least = INFINITY, most = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < live) least = fminf(least, gb[i]), most = fmaxf(most, gb[i]);
        const float f = scale_shift(ga_lane, least, most);
        ga_lane *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) gb[i] /= f;
    }
#pragma unroll 2
    for (int i = 0; i < (NT + WARPS - 1) / WARPS; ++i) {
        const int c = c0 + splits * WARPS * i;
        const float a = __shfl_sync(0xffffffffu, ga_lane, i);
        if (c >= rows) break;
        const float* p = part + c * 128 + 4 * lane;
        float4 v = splits > 1 ? ld_peer_f4(p, 0) : *reinterpret_cast<const float4*>(p);
        for (int r = 1; r < splits; ++r) {
            const float4 o = ld_peer_f4(p, r);
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        const float f[4] = {v.x * a * gb[0], v.y * a * gb[1], v.z * a * gb[2], v.w * a * gb[3]};
        T* y = static_cast<T*>(args.y) + (m0 + c) * args.ldy + n;
        if (wide && live == 4) {
            __align__(16) T o[4] = {out_value<T>(f[0]), out_value<T>(f[1]), out_value<T>(f[2]), out_value<T>(f[3])};
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(o);
            else *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(o);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < live) y[j] = out_value<T>(f[j]);
        }
    }
}

// Grid: x = weight tile * splits + rank (a cluster of `splits` CTAs per tile), y = tile of NT activation rows.
template <int NT, typename T>
__global__ void __launch_bounds__(kRowsThreads, 1)
    nvfp4_rows_matmul_kernel(const __grid_constant__ MatmulArgs args, const int splits) {
    constexpr int kStages = rows_stages<NT>(), kStageBytes = rows_stage_bytes<NT>();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = splits > 1 ? (int)cluster_rank() : 0;
    const int64_t nt = blockIdx.x / splits, m0 = (int64_t)blockIdx.y * NT;
    const int k0 = (int)((int64_t)args.KT * rank / splits), k1 = (int)((int64_t)args.KT * (rank + 1) / splits);

    // the weights and the activations of K step kt into stage s
    auto load_w = [&](int s, int kt) {
        unsigned char* p = smem + (size_t)s * kStageBytes;
        const size_t at = (size_t)nt * args.KT + kt;
        bulk_load(p, args.qb + at * kTile, kTile, &full[s]);
        bulk_load(p + kTile + NT * 128, args.sb + at * kAtoms * kAtom, kAtoms * kAtom, &full[s]);
    };
    auto load_x = [&](int s, int kt) {
        unsigned char* p = smem + (size_t)s * kStageBytes;
        const size_t at = (size_t)(m0 / 128) * args.KT + kt;
        bulk_load(p + kTile, args.qa + at * kTile + (m0 % 128) * 128, NT * 128, &full[s]);
        bulk_load(p + kTile + NT * 128 + kAtoms * kAtom, args.sa + at * kAtoms * kAtom, kAtoms * kAtom, &full[s]);
    };
    const int head = min(kStages, k1 - k0);
    if (warp == 0 && elect_one()) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        // at once, if they may: the rest of the set-up runs meanwhile
        if (!args.weights_ready) pdl_wait();
        for (int it = 0; it < head; ++it) {
            mbar_arrive_expect_tx(&full[it], kStageBytes);
            load_w(it, k0 + it);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr uint32_t kSfBase = NT;  // scale columns after the accumulator

    if (warp == 0) {
        if (elect_one()) {
            int it = head;
            pdl_wait();
            for (int i = 0; i < head; ++i) load_x(i, k0 + i);
            for (; it < k1 - k0; ++it) {
                const int s = it % kStages;
                if (!mbar_wait(&empty[s], ((it / kStages) & 1) ^ 1, abort_flag, args.status)) break;
                mbar_arrive_expect_tx(&full[s], kStageBytes);
                load_w(s, k0 + it);
                load_x(s, k0 + it);
            }
            land(full, it, kStages);
        }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_mxf4nvf4_ue4m3(128, NT);
        for (int it = 0; it < k1 - k0; ++it) {
            const int s = it % kStages;
            if (!mbar_wait_warp(&full[s], (it / kStages) & 1, abort_flag, args.status)) break;
            tc_fence_after();
            unsigned char* p = smem + (size_t)s * kStageBytes;
            unsigned char* sf = p + kTile + NT * 128;
            rows_stage_mma(tmem, tmem + kSfBase + s * 32, desc_sw128(p), desc_sw128(p + kTile), desc_sf(sf),
                           desc_sf(sf + kAtoms * kAtom), idesc, it > 0 ? 1u : 0u, &empty[s]);
        }
        // fires once every MMA and scale copy of this warp has completed (also when aborting)
        tc_commit(acc_full);
    }
    __syncwarp();
    pdl_wait();  // ga comes from the kernel before
    pdl_launch_dependents();
    volatile int never = 0;
    mbar_wait(acc_full, 0, &never, args.status);  // the commit always comes; bounded all the same
    tc_fence_after();
    __syncthreads();  // and no copy is in flight: they have landed, or (bounded) been waited for

    // Results go through shared memory, [activation row][128 weight rows], on the stages; activation row c of the tile is
    // then summed over the cluster's CTAs, in rank order, scaled and stored by a warp of CTA c % splits.
    float* part = reinterpret_cast<float*>(smem);
    const int rows = (int)min((int64_t)NT, args.M - m0);
    if (warp >= 2) {
        const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll 1
        for (int c = 0; c < rows; c += 8) {
            uint32_t v[8];
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                         : "r"(acc + c));
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) part[(c + i) * 128 + 32 * (warp & 3) + lane] = __uint_as_float(v[i]);
        }
    }
    __syncwarp();
    if (splits > 1) cluster_sync();
    else __syncthreads();
    store_rows<T, kRowsThreads / 32, NT>(args, part, nt, m0, rows, rank, splits, args.ga + (args.ga_rows ? m0 : 0), args.ga_rows != 0);
    if (splits > 1) {
        __syncwarp();
        cluster_sync();  // the partial sums stay until every CTA has read them
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ------------------------------------------------------------------ pair kernel
// Two CTAs (a cluster, two neighbouring SMs) share one 256 x 256 tile (cta_group::2): CTA r holds the tile's A rows
// 128 r .. and B rows 128 r .. in shared memory and A rows' results (128 lanes x 256 columns) in its tensor
// memory; the leader (rank 0) issues the MMAs of both.  Each CTA thus copies 32 KB of codes per K step for
// 128 x 256 results instead of 48 KB.  The scales of all 256 B rows go to both CTAs' tensor memory.
//   warp 0     copies this CTA's operands (tensor copies, whose bytes the leader's barrier counts)
//   warp 1     rank 0: waits for a stage of both CTAs, issues scale copies and MMAs, whose commit frees the stage
//              in both
//   warps 2-9  epilogue: two warps per lane quarter, each half of the columns; registers first, so that the next
//              tile's MMAs run while these values are scaled and stored
constexpr int kPairStages = 5;
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int kPairStageBytes = 2 * kTile + 12 * kAtom;  // A, B, A's scales, both halves of B's scales
constexpr int kPairSfCols = 48;
constexpr uint32_t kPairSfBase = 256;  // scale columns after the accumulator
constexpr int kTurnWords = 32 * 17;  // a warp's 32 rows of 64 bytes, one word of padding each
constexpr size_t kPairSmem = (size_t)kPairStages * kPairStageBytes + (512 + 4 * kTurnWords) * kPairEpiWarps + 1024 + 256;
static_assert(kPairStageBytes % 1024 == 0 && kPairSfBase + kPairStages * kPairSfCols <= kTmemCols, "stage alignment, tensor memory");
static_assert(kPairSmem <= 232448, "shared memory");

// The high words of the matrix descriptors of tcgen05.cuh (desc_sw128, desc_sf); the low one is address / 16 | 2^16.
constexpr uint32_t kSw128High = (1024 >> 4) | (1u << 14) | (2u << 29), kSfHigh = (128 >> 4) | (1u << 14);

// One K step of a pair, by one thread: as stage_scales_nv_to_tmem and stage_mmas_nv_commit (tcgen05.cuh), with copies that run in
// both CTAs and a commit that arrives on the barrier at this offset in both.  a, b, sa, sb0, sb1: low words.  The step's
// latency is part of a stage's round trip, so that descriptors are built from 32-bit words, by one thread without a vote.
__device__ __forceinline__ void pair_scales(uint32_t sf, uint32_t sa, uint32_t sb0, uint32_t sb1) {
    asm volatile(
        "{\n\t.reg .b32 c, l;\n\t.reg .b64 t;\n\t"
#define COPY(column, low, atom)                                                             \
    "add.u32 c, %0, " #column ";\n\tadd.u32 l, " low ", " #atom ";\n\tmov.b64 t, {l, %4};\n\t" \
    "tcgen05.cp.cta_group::2.32x128b.warpx4 [c], t;\n\t"
        COPY(0, "%1", 0) COPY(16, "%2", 0) COPY(20, "%3", 0) COPY(4, "%1", 32) COPY(24, "%2", 32) COPY(28, "%3", 32)
        COPY(8, "%1", 64) COPY(32, "%2", 64) COPY(36, "%3", 64) COPY(12, "%1", 96) COPY(40, "%2", 96) COPY(44, "%3", 96)
#undef COPY
        "}" ::"r"(sf), "r"(sa), "r"(sb0), "r"(sb1), "n"(kSfHigh)
        : "memory");
}
__device__ __forceinline__ void pair_products(uint32_t d, uint32_t sf, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate,
                                              uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b16 both;\n\t.reg .b32 c, e, l, m;\n\t.reg .b64 t, u;\n\t"
        "mov.b16 both, 3;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.eq.b32 q, %5, %5;\n\t"
#define PRODUCT(i, pred)                                                                                   \
    "add.u32 l, %1, 2*" #i ";\n\tadd.u32 m, %2, 2*" #i ";\n\tmov.b64 t, {l, %7};\n\tmov.b64 u, {m, %7};\n\t" \
    "add.u32 c, %4, 4*" #i ";\n\tadd.u32 e, %4, 16+8*" #i ";\n\t"                                          \
    "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], t, u, %3, [c], [e], " pred ";\n\t"
        PRODUCT(0, "p") PRODUCT(1, "q") PRODUCT(2, "q") PRODUCT(3, "q")
#undef PRODUCT
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%6], both;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sf), "r"(accumulate), "r"(bar), "n"(kSw128High)
        : "memory");
}
__device__ __forceinline__ void pair_commit(uint64_t* bar) {  // by one thread
    asm volatile(
        "{\n\t.reg .b16 both;\n\t"
        "mov.b16 both, 3;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
// A box of whole 1 KB rows of an operand's bytes (the map: [bytes / 1024][256 words]) into this CTA's shared memory; the bytes
// are counted on a barrier of the leader.
__device__ __forceinline__ void pair_load(void* dst, const CUtensorMap* map, int64_t at, uint32_t leader_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(0), "r"((int)(at / 1024)), "r"(leader_bar)
        : "memory");
}
__device__ __forceinline__ uint32_t leader_address(const void* p) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
// Arrive on the barrier at this offset in CTA 0 of the cluster.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
// 64 bytes (`left` elements or more) of each of a warp's 32 rows (those below `rows`) from shared memory to y, row by row, a word
// per lane.  Out of line: the epilogue's code has to stay small, or it waits for its instructions.
template <typename T>
__device__ __noinline__ void store_ragged(const uint32_t* turn, T* y, int64_t ldy, int rows, int left) {
    constexpr int kPerWord = 4 / (int)sizeof(T);
    const int lane = threadIdx.x & 31, r0 = lane >> 4;
    left -= kPerWord * (lane & 15);
    T* to = y + r0 * ldy + kPerWord * (lane & 15);
#pragma unroll 4
    for (int i = 0; i < 16; ++i, to += 2 * ldy) {
        const uint32_t w = turn[17 * (2 * i + r0) + (lane & 15)];
        if (2 * i + r0 >= rows || left <= 0) continue;
        if (sizeof(T) == 4 || (left > 1 && reinterpret_cast<uintptr_t>(to) % 4 == 0)) {
            *reinterpret_cast<uint32_t*>(to) = w;
        } else {
            reinterpret_cast<uint16_t*>(to)[0] = (uint16_t)w;
            if (left > 1) reinterpret_cast<uint16_t*>(to)[1] = (uint16_t)(w >> 16);
        }
    }
}
struct PairArgs {
    CUtensorMap qa, sa, qb, sb;  // the operands' bytes in rows of 1 KB
    MatmulArgs m;
};

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    nvfp4_pair_matmul_kernel(const __grid_constant__ PairArgs pair, const int MT, const int NT) {
    const MatmulArgs& args = pair.m;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* gb_smem = reinterpret_cast<float*>(smem + kPairStages * kPairStageBytes);  // [epilogue warp][128]
    uint32_t* turn_smem = reinterpret_cast<uint32_t*>(gb_smem + 128 * kPairEpiWarps);  // [epilogue warp][32][17]
    uint64_t* full = reinterpret_cast<uint64_t*>(turn_smem + kTurnWords * kPairEpiWarps);  // rank 0: the copies of both CTAs
    uint64_t* empty = full + kPairStages;
    uint64_t* acc_full = empty + kPairStages;
    uint64_t* acc_empty = acc_full + 1;  // rank 0: the epilogue warps of both CTAs
    uint64_t* mma_done = acc_empty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 2 * kPairEpiWarps);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const int n_tiles = MT * NT, KT = args.KT, first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int64_t last_a = (args.M + 127) / 128 - 1, last_b = (args.N + 127) / 128 - 1;  // last 128-row blocks
    auto stage = [&](int s) { return smem + (size_t)s * kPairStageBytes; };

    if (warp == 0) {
        if (elect_one()) {
            int it = 0;
            bool ok = true;
            for (int t = first; t < n_tiles && ok; t += step) {
                const int64_t ab = min(2 * (int64_t)(t / NT) + rank, last_a), b0 = 2 * (int64_t)(t % NT), b1 = min(b0 + 1, last_b);
                const size_t ka = (size_t)ab * KT, kb0 = (size_t)b0 * KT, kb1 = (size_t)b1 * KT, kb = rank == 0 ? kb0 : kb1;
                for (int kt = 0; kt < KT; ++kt, ++it) {
                    const int s = it % kPairStages;
                    if (!mbar_wait(&empty[s], ((it / kPairStages) & 1) ^ 1, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    unsigned char* p = stage(s);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPairStageBytes);
                    const uint32_t bar = leader_address(&full[s]);
                    pair_load(p, &pair.qa, (ka + kt) * kTile, bar);
                    pair_load(p + kTile, &pair.qb, (kb + kt) * kTile, bar);
                    pair_load(p + 2 * kTile, &pair.sa, (ka + kt) * kAtoms * kAtom, bar);
                    pair_load(p + 2 * kTile + 4 * kAtom, &pair.sb, (kb0 + kt) * kAtoms * kAtom, bar);
                    pair_load(p + 2 * kTile + 8 * kAtom, &pair.sb, (kb1 + kt) * kAtoms * kAtom, bar);
                }
            }
            // The leader's barriers count the copies of both CTAs.
            if (rank == 0) land(full, it, kPairStages);
        }
    } else if (warp == 1 && rank == 0) {
        if (elect_one()) {
            const uint32_t idesc = idesc_mxf4nvf4_ue4m3(256, 256), base = smem_u32(smem);
            int s = 0, tile = 0;
            uint32_t phase = 0;
            bool ok = true;
            // waits for a stage and sends its scales to tensor memory
            auto scales = [&]() {
                if (!mbar_wait(&full[s], phase, abort_flag, args.status)) return false;
                tc_fence_after();
                const uint32_t sf = ((base + s * kPairStageBytes + 2 * kTile) >> 4) | (1u << 16);
                pair_scales(tmem + kPairSfBase + s * kPairSfCols, sf, sf + 4 * kAtom / 16, sf + 8 * kAtom / 16);
                return true;
            };
            auto products = [&](uint32_t accumulate) {
                const uint32_t p = ((base + s * kPairStageBytes) >> 4) | (1u << 16);
                pair_products(tmem, tmem + kPairSfBase + s * kPairSfCols, p, p + kTile / 16, idesc, accumulate, smem_u32(&empty[s]));
                if (++s == kPairStages) s = 0, phase ^= 1;
            };
            for (int t = first; t < n_tiles && ok; t += step, ++tile) {
                // (the first step's scales while the results of the tile before are read)
                if (!scales() || !mbar_wait(acc_empty, (tile & 1) ^ 1, abort_flag, args.status)) break;
                tc_fence_after();
                products(0u);
                for (int kt = 1; kt < KT; ++kt) {
                    if (!scales()) {
                        ok = false;
                        break;
                    }
                    products(1u);
                }
                if (ok) pair_commit(acc_full);
            }
            pair_commit(mma_done);
        }
        __syncwarp();
    } else if (warp >= 2) {
        const int q = warp & 3, half = (warp - 2) / 4;
        const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + 128 * half;
        const bool wide = reinterpret_cast<uintptr_t>(args.y) % 16 == 0 && (args.ldy * (int64_t)sizeof(T)) % 16 == 0;
        float* gb = gb_smem + 128 * (warp - 2);
        uint32_t* turn = turn_smem + kTurnWords * (warp - 2);
        T* y = static_cast<T*>(args.y);
        int tile = 0;
        for (int t = first; t < n_tiles; t += step, ++tile) {
            const int64_t m0 = (int64_t)(t / NT) * 256 + 128 * rank + 32 * q, n0 = (int64_t)(t % NT) * 256 + 128 * half;
            const int64_t m = m0 + lane;
            float ga = m < args.M ? args.ga[args.ga_rows ? m : 0] : 1.f;
            const int live = (int)max((int64_t)0, min((int64_t)128, args.N - n0));  // columns of this warp's half
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (32 * c + lane < live) gb[32 * c + lane] = args.gb[args.gb_rows ? n0 + 32 * c + lane : 0];
            __syncwarp();
            if (__any_sync(0xffffffffu, far_scale(ga))) {
                float least = INFINITY, most = 0.f;
                for (int i = lane; i < live; i += 32) least = fminf(least, gb[i]), most = fmaxf(most, gb[i]);
                const float f = scale_shift(ga, least, most);
                ga *= f;
                for (int i = lane; i < live; i += 32) gb[i] /= f;
                __syncwarp();
            }
            if (!mbar_wait(acc_full, tile & 1, abort_flag, args.status)) break;
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(acc + 32 * c, v[c]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(acc_empty);
            // 16-byte pieces transposed inside groups of four lanes: a store writes 64 contiguous bytes of 8 rows
            const int64_t r0 = m0 + 4 * (lane >> 2);
            T* out = y + r0 * args.ldy + n0 + (lane & 3) * (16 / (int)sizeof(T));
            const int rows = (int)max((int64_t)0, min((int64_t)4, args.M - r0));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (32 * c >= live) break;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 g = *reinterpret_cast<const float4*>(gb + 32 * c + i);
                    v[c][i] = __float_as_uint(__uint_as_float(v[c][i]) * ga * g.x);
                    v[c][i + 1] = __float_as_uint(__uint_as_float(v[c][i + 1]) * ga * g.y);
                    v[c][i + 2] = __float_as_uint(__uint_as_float(v[c][i + 2]) * ga * g.z);
                    v[c][i + 3] = __float_as_uint(__uint_as_float(v[c][i + 3]) * ga * g.w);
                }
                if (wide && 32 * c + 32 <= live) {
                    constexpr int kHalves = (int)sizeof(T) / 2;  // 32 columns: one or two times 64 bytes
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        uint4 pc[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) pc[p] = out_piece<T>(&v[c][(32 / kHalves) * h + (16 / (int)sizeof(T)) * p]);
                        transpose4_pieces(pc, lane);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < rows) *reinterpret_cast<uint4*>(out + j * args.ldy + 32 * c + (32 / kHalves) * h) = pc[j];
                    }
                } else {
                    // rows that do not start on 16 bytes, or the ragged last columns: 64 bytes of each of the warp's 32 rows
                    // through shared memory, then stored row by row, a word per lane
                    constexpr int kHalves = (int)sizeof(T) / 2;
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const uint4 o = out_piece<T>(&v[c][(32 / kHalves) * h + (16 / (int)sizeof(T)) * p]);
                            uint32_t* to = turn + 17 * lane + 4 * p;
                            to[0] = o.x, to[1] = o.y, to[2] = o.z, to[3] = o.w;
                        }
                        __syncwarp();
                        const int col = 32 * c + (32 / kHalves) * h;
                        store_ragged<T>(turn, y + m0 * args.ldy + n0 + col, args.ldy, (int)min((int64_t)32, args.M - m0), live - col);
                        __syncwarp();
                    }
                }
            }
            __syncwarp();  // gb is rewritten for the next tile
        }
    }
    __syncwarp();
    {
        // every MMA and scale copy has completed: the leader commits mma_done last, aborting or not
        volatile int never = 0;
        mbar_wait(mma_done, 0, &never, nullptr);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA's shared or tensor memory goes while the other may use it
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ------------------------------------------------------------------ host side
// CTAs that share a tile's K range: more while the tiles leave SMs idle and every CTA keeps at least two K steps.
int k_splits(int64_t tiles, int KT) {
    int splits = 1;
    while (splits < 8 && tiles * splits * 2 <= sm_count() && KT / (splits * 2) >= 2) splits *= 2;
    return splits;
}

template <int NT>
cudaError_t launch_rows(const MatmulArgs& a, cudaStream_t st) {
    const int64_t wt = (a.N + 127) / 128, mt = (a.M + NT - 1) / NT;
    int splits = k_splits(wt * mt, a.KT);
    const void* f = a.dtype == MOE_F32    ? (const void*)nvfp4_rows_matmul_kernel<NT, float>
                    : a.dtype == MOE_BF16 ? (const void*)nvfp4_rows_matmul_kernel<NT, __nv_bfloat16>
                                          : (const void*)nvfp4_rows_matmul_kernel<NT, __half>;
    void* args[] = {const_cast<MatmulArgs*>(&a), &splits};
    return launch_cluster(f, dim3((unsigned)(wt * splits), (unsigned)mt), kRowsThreads, rows_smem<NT>(), splits, st, args);
}

// Map of `bytes` bytes as rows of 1 KB, read in boxes of `box` bytes (both multiples of 1 KB).
cudaError_t byte_map(CUtensorMap* m, const uint8_t* p, int64_t bytes, int box) {
    encode_tiled_fn enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {256, (cuuint64_t)(bytes / 1024)};
    const cuuint64_t strides[1] = {1024};
    const cuuint32_t boxes[2] = {256, (cuuint32_t)(box / 1024)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(p), dims, strides, boxes, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_nvfp4_matmul(const moe_nvfp4_operand* A, const moe_nvfp4_operand* B, int64_t M, int64_t N, int64_t K, void* y,
                                moe_dtype dtype, int64_t ldy, int* status, cudaStream_t st, bool weights_ready) {
    if (M == 0 || N == 0) return cudaSuccess;
    MatmulArgs a = {A->q, A->s, A->gs, A->gs_rows, B->q, B->s, B->gs, B->gs_rows, M, N, (int)((K + 255) / 256), y, (int)dtype, ldy,
                    status, weights_ready ? 1 : 0};
    if (M <= 8) return launch_rows<8>(a, st);
    if (M <= 16) return launch_rows<16>(a, st);
    if (M <= 32) return launch_rows<32>(a, st);
    if (M <= 64) return launch_rows<64>(a, st);
    // Beyond 128 rows the pair kernel's tiles are few and large: while one wave of 128 x 128 tiles (their K range split over a
    // cluster where they leave SMs idle) covers the results, these finish sooner, unless K is so short that the fixed costs
    // decide (us, rows / pair: 256 x 4096 x 8192 11.1 / 14.5, 512 x 4096 x 8192 13.4 / 15.5, 256 x 8192 x 4096 10.0 / 10.9, 777 x
    // 1000 x 1544 8.0 / 8.4; beyond a wave, 512 x 8192 x 1024 13.3 / 7.7; short K, 1024^3 7.4 / 7.1, 200 x 600 x 300 6.6 / 6.3).
    if (M <= 128 || (a.KT > 4 && ((M + 127) / 128) * ((N + 127) / 128) <= sm_count())) return launch_rows<128>(a, st);
    int MT = (int)((M + 255) / 256), NT = (int)((N + 255) / 256);
    const int64_t tiles = (int64_t)MT * NT, pairs = sm_count() / 2;
    PairArgs p;
    p.m = a;
    const int64_t Kp = (int64_t)a.KT * 256, Mp = (M + 127) / 128 * 128, Np = (N + 127) / 128 * 128;
    cudaError_t e = byte_map(&p.qa, A->q, Mp * Kp / 2, kTile);
    if (e == cudaSuccess) e = byte_map(&p.sa, A->s, Mp * Kp / 16, kAtoms * kAtom);
    if (e == cudaSuccess) e = byte_map(&p.qb, B->q, Np * Kp / 2, kTile);
    if (e == cudaSuccess) e = byte_map(&p.sb, B->s, Np * Kp / 16, kAtoms * kAtom);
    if (e != cudaSuccess) return e;
    void* args[] = {&p, &MT, &NT};
    const void* f = dtype == MOE_F32    ? (const void*)nvfp4_pair_matmul_kernel<float>
                    : dtype == MOE_BF16 ? (const void*)nvfp4_pair_matmul_kernel<__nv_bfloat16>
                                        : (const void*)nvfp4_pair_matmul_kernel<__half>;
    return launch_kernel(f, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kPairThreads), kPairSmem, st, true, args);
}

}  // namespace moe
