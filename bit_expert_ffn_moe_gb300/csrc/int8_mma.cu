// int8_mma.cu -- the 8-bit products on the tensor cores.  sm_103a's have no 8-bit whole numbers, but numbers up to 2048 are exact in fp16,
// their products exact and sums too as long as they stay within 2^24: so kind::f16, at the rate of bf16.
//   The weights are the MMA's M side (128 weight rows a CTA) and come from tensor memory: read as bytes, turned into fp16 in
// registers by sixteen warps, stored to tensor memory, so that they cost one byte of memory traffic and shared memory sees them
// once.  The activations are the N side (16 .. 192 rows), fp16 already, copied as they lie.
//   warps 0-15   conversion: four sets of four warps, each a quarter of the tiles of 64 values
//   warps 16-19  epilogue: accumulators (two, so that the next tile's products run meanwhile), scales, store; of the CTA's last
//                part all twenty warps (1024 x 4096 x 8192: 76 us with four, 59 with twenty)
//   warp 20      copies of weights, one a step of 128 values; a step's place is free once it is converted
//   warp 21      copies of activations, two a step; a step's place is free once its products are done
//   warp 22      products
// (Weights come from memory and activations mostly from L2, so weights have the longer ring.  With one ring for both, the gate and up
// products of 256 tokens by 8 of 128 experts of 8192 x 2048 took 687 us instead of 652, of 4096 tokens 1454 instead of 1396.)
// PAIR: two CTAs share a tile of 256 weight rows (cta_group::2), each with half of the activation rows in its shared memory; the
// leader (rank 0) issues the products of both, and the other's warp 22 passes on that its activations are there.
// Work: the tiles of all experts in a row, taken in turns; the last ones, where it saves enough, are dealt out by their steps.  A tile that
// several CTAs share is summed by the last of them to arrive, from partial sums in memory, in the order of the CTAs.
// 736 threads leave 80 registers each, and some 50 words are spilled -- none in the loops over the steps: a launch of 4096 x 4096 x 2048, 4096
// or 8192 makes the same 82536 local loads of a warp, 24 of each.
// Every barrier wait is bounded: on expiry the CTA records MOE_ERR_TIMEOUT, waits (bounded) for its own copies and products,
// frees tensor memory and exits.
#include "int8_mma.cuh"

namespace moe {
namespace {

constexpr int kSets = 4, kConvWarps = 4 * kSets, kEpiWarps = 4, kFinishWarps = kConvWarps + kEpiWarps;
constexpr int kWeightWarp = kFinishWarps, kRowWarp = kWeightWarp + 1, kMmaWarp = kRowWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kMostRows = 192;       // activation rows of a tile
constexpr int kMostStages = 16;
// A step is two tiles of weights, 128 values (the last one of an odd number of tiles: one).  The converted weights of a tile are a slot in
// tensor memory; set i of the converting warps fills slot i, with tile i % 2 of every other step.
constexpr uint32_t kTmemCols = 512, kSlotCols = 32, kSlotBase = 2 * kMostRows;
static_assert(kSlotBase + kSets * kSlotCols == kTmemCols, "tensor memory");
// Steps that a CTA's share of split tiles has at least, and that splitting has to save: bringing the sums together costs some 10 us.  (512 x 8192
// x 8192: 73 us with 8, 58.5 with 32, 62 without; 1024 x 8192 x 4096: 64, 50.5, 50.5; 2048 x 4096 x 8192: 90, 88, 92.)
constexpr int kLeastSteps = 32;
constexpr size_t kSmemMost = 232448;
constexpr int kStepBytes = 2 * kInt8Tile;  // of weights

struct Shared {
    uint64_t w_full[kMostStages], w_empty[kMostStages], x_full[kMostStages], x_empty[kMostStages], ready[kMostStages], acc_full[2], acc_empty[2], epilogue, all, parts, done;
    uint32_t tmem;
    volatile int abort;
    int last[3];  // whether this CTA is the last to arrive at a shared tile: at the one before the last, or the last
    int split, ctas, whole;  // tiles that CTAs (PAIR: pairs) share, how many of these do, and tiles that one CTA computes
    alignas(16) float sx[kEpiWarps + 1][kMostRows];  // scales of the rows of the epilogue's warps' tiles; of the last part
    int32_t tiles[kMaxE + 1], offset[kMaxE + 1];  // tiles and rows of the experts before
};

struct MmaArgs {
    Int8ProductArgs p;
    int most, x_bytes;       // activation rows of a tile at most; their bytes a tile of weights
    int w_steps, x_steps;    // steps in the ring of weights, and behind it in that of activations; even numbers
    int slot_rows;  // of partial sums, a multiple of 16
};

__host__ __device__ __forceinline__ int ring_bytes(const MmaArgs& m) { return m.w_steps * kStepBytes + m.x_steps * 2 * m.x_bytes; }

// An expert's rows as mt tiles of up to n rows (a multiple of 16).
struct Rows {
    int64_t count;
    int mt, n;
};
__device__ __forceinline__ Rows rows_of(int64_t count, int most) {
    Rows r;
    r.count = count;
    r.mt = (int)((count + most - 1) / most);
    r.n = count > 0 ? ((int)((count + r.mt - 1) / r.mt) + 15) / 16 * 16 : 16;
    return r;
}

// Steps k .. k1 - 1 of a tile: of expert e, its weight tile nt and activation tile mt.
struct Part {
    int id, e, nt, mt, k, k1;  // id: among all tiles (M N is at most 2^40: they fit)
    bool last;                 // of the CTA
    Rows r;
};

// The tiles of all experts in a row, expert by expert, weight tile by weight tile.  CTAs take them in turns, so that at any time
// neighbours work on the same weights and rows, which then come out of L2 (contiguous shares: each tile's operands from memory, 2.7
// ms instead of 1.5 for the gate and up products of 4096 tokens).  The last `split` of them, fewer than there are CTAs, are dealt
// out by their steps, evenly, so that all CTAs end at the same time.  (Shared tiles first, their sums made while the next
// tile's products run: the sums' loads waited behind the copies for longer than that tile took, 94 us instead of 59 for 1024 x 4096 x 8192.)
template <bool PAIR>
struct Work {
    const Shared& s;
    const int64_t M;  // rows of a dense product (by expert: -1)
    const int NT, E, KS, most, G;  // weight tiles (PAIR: of 256 rows), experts, steps of a tile, CTAs

    __device__ __forceinline__ Work(const Shared& shared, const MmaArgs& args)
        : s(shared), M(args.p.offsets ? -1 : args.p.M), NT((int)((args.p.N + (PAIR ? 255 : 127)) / (PAIR ? 256 : 128))), E(args.p.E),
          KS((int)((args.p.K + 127) / 128)), most(args.most), G(PAIR ? (int)gridDim.x / 2 : (int)gridDim.x) {}

    __device__ __forceinline__ Rows rows(int e) const { return rows_of(M >= 0 ? M : s.offset[e + 1] - s.offset[e], most); }
    // The first step of CTA c's share of the split tiles.  (32 bits: fewer tiles than CTAs, 1024 steps a tile at most.)
    __device__ __forceinline__ int share(int c) const { return (int)((unsigned)(s.split * KS) * (unsigned)c / (unsigned)s.ctas); }
    // The CTAs that share tile `id`: those whose shares have its first step and its last one.  (share(c) <= u where split KS c < (u + 1) ctas.)
    __device__ __forceinline__ void sharers(int id, int& first, int& last) const {
        const unsigned all = s.split * KS, b = (id - s.whole) * KS;
        first = (int)(((b + 1) * (unsigned)s.ctas - 1) / all);
        last = (int)(((b + KS) * (unsigned)s.ctas - 1) / all);
    }
    // CTA c's last part, and its number among the CTA's parts (-1: no work).
    __device__ __forceinline__ int last(int c, Part& p) const {
        int number = c < s.whole ? (s.whole - 1 - c) / G : -1;  // of its whole tiles' last one
        p.id = c + number * G;
        p.k = 0, p.k1 = KS;
        if (c < s.ctas) {
            const int u = share(c), end = share(c + 1), tile = (end - 1) / KS;
            number += tile - u / KS + 1;
            p.id = s.whole + tile;
            p.k = max(0, u - tile * KS);
            p.k1 = end - tile * KS;
        }
        if (number < 0) return -1;
        p.last = true;
        place(p, -1);
        return number;
    }
    // Expert and tiles of p.id; e: an expert before its.
    __device__ __forceinline__ void place(Part& p, int e) const {
        if (e < 0 || s.tiles[e + 1] <= p.id) {
            do ++e;
            while (s.tiles[e + 1] <= p.id);
            p.r = rows(e);
        }
        p.e = e;
        const int tile = p.id - s.tiles[e];
        p.nt = tile / p.r.mt;
        p.mt = tile - p.nt * p.r.mt;
    }
    // f(part) for CTA c's work, until it returns false.
    template <typename F>
    __device__ __forceinline__ void each(int c, F f) const {
        Part p;
        p.e = -1;
        int left = 0, k = 0, id = c, shared = 0;  // steps of the share; its first, and its first tile
        if (c < s.ctas) {
            const int u = share(c);
            left = share(c + 1) - u;
            shared = u / KS;
            k = u - shared * KS;
            shared += s.whole;
        }
        while (true) {
            p.k = 0, p.k1 = KS;
            if (id < s.whole) {
                p.id = id;
                id += G;
            } else {
                if (left <= 0) return;
                p.id = shared++;
                p.k = k;
                p.k1 = min(KS, k + left);
                left -= p.k1 - k;
                k = 0;
            }
            p.last = left <= 0 && id >= s.whole;
            place(p, p.e);
            if (!f(p)) return;
        }
    }
};

// Activation rows of a tile, rounded up to 16.
__device__ __forceinline__ int tile_rows(const Part& p) {
    return min(p.r.n, ((int)min((int64_t)kMostRows, p.r.count - (int64_t)p.mt * p.r.n) + 15) / 16 * 16);
}
__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Results of the CTA's part p, its tile number `tile`: this warp's lane quarter, units of 16 activation rows unit0, unit0 + stride, ...
// sx: room for the rows' scales, of this warp or with the same from others; verdict: a word of the warps that sync() brings together.
template <typename T, bool GATED, bool PAIR, typename Sync>
__device__ __forceinline__ bool finish(const MmaArgs& args, Shared& s, unsigned char* ring, const Work<PAIR>& work, uint32_t tmem, const Part& p, int tile,
                                       int unit0, int stride, float* sx, volatile int* verdict, Sync sync) {
    const Int8ProductArgs& a = args.p;
    const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3, b = tile & 1;
    const int rank = PAIR ? (int)cluster_rank() : 0, cta = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x;
    const bool speaker = threadIdx.x == 32 * kConvWarps;
    int* const status = &a.ctrl->status;
    const int64_t m0 = (int64_t)p.mt * p.r.n;
    const int live = (int)min((int64_t)p.r.n, p.r.count - m0);
    const int n0 = (PAIR ? 2 * p.nt + rank : p.nt) * 128 + 32 * q, n = n0 + lane, N = (int)a.N;  // (N is at most 2^28)
    const float sw = n < N ? __ldg(a.sw + (int64_t)p.e * a.N + n) : 0.f;
    const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + b * kMostRows;
    {
        const float* const from = a.sx + (a.offsets ? int8_first_row(s.offset[p.e], p.e) : 0) + m0;
        __syncwarp();
#pragma unroll
        for (int c0 = 0; c0 < kMostRows; c0 += 32)
            if (c0 + lane < live) sx[c0 + lane] = __ldcg(from + c0 + lane);
    }
    // The CTA's last part: all of its products are done.  (Not its accumulators' phase: the converting warps have not waited for all the
    // phases before it, and a parity does not tell a phase from the one before the last.)
    if (!mbar_wait_warp(p.last ? &s.done : &s.acc_full[b], p.last ? 0 : (tile >> 1) & 1, &s.abort, status)) return false;
    if (p.last && __any_sync(0xffffffffu, s.abort)) return false;
    tc_fence_after();
    int first = cta, last = cta;  // the CTAs that share the tile
    // The partial sums of a CTA, [16 activation rows][4][128][4]: of the tile that it begins, or (1) goes on with.
    auto slot = [&](int c) {
        return reinterpret_cast<float4*>(a.partials + (((int64_t)c * (PAIR ? 2 : 1) + rank) * 2 + (c > first)) * 128 * args.slot_rows);
    };
    if (p.k > 0 || p.k1 < work.KS) {
        work.sharers(p.id, first, last);
        unsigned* const count = &a.ctrl->int8_split[first * (PAIR ? 2 : 1) + rank];
        // the last CTA to arrive adds the others' sums to its own; where the others are there already, it need not store them
        if (speaker) *verdict = ld_acquire(count) == (unsigned)(last - first);
        if (!sync()) return false;
        bool mine = *verdict != 0;
        if (!mine) {
            for (int c0 = 16 * unit0; c0 < live; c0 += 16 * stride) {  // (slots have room for whole sixteens)
                float4* const to = slot(cta) + c0 * 32 + 32 * q + lane;
                uint32_t v[16];
                tmem_ld16(acc + c0, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    __stcg(to + i * 128, make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                                                     __uint_as_float(v[4 * i + 3])));
            }
            __threadfence();
            if (!sync()) return false;
            if (speaker) {
                *verdict = atomicAdd(count, 1u) == (unsigned)(last - first);
                __threadfence();
            }
            if (!sync()) return false;
            mine = *verdict != 0;
        }
        if (!mine) return true;
        if (speaker) *count = 0;  // (every one of them has arrived)
    }
    const bool odd = lane & 1, whole = n0 + 32 <= N;
    const bool pairs = sizeof(T) == 2 && reinterpret_cast<uintptr_t>(a.y) % 4 == 0 && a.ldy % 2 == 0;
    T* const out = static_cast<T*>(a.y) + ((a.offsets ? s.offset[p.e] : 0) + m0) * a.ldy +
                   (GATED ? odd * a.ldy + n / 2 : pairs ? odd * a.ldy + (n & ~1) : (int64_t)n);
    // Others' sums: in the CTA's last part (most often it is that) through the ring, which nothing uses any more, as many rows at a
    // time as fit; else straight from memory.
    const int others = last - first, ring_rows = p.last && others > 0 ? ring_bytes(args) / (others * 512) / 16 * 16 : 0;
    uint32_t parts = 0;
    for (int begin = 0, end; begin < live; begin = end) {
        end = ring_rows > 0 ? min(begin + ring_rows, (live + 15) / 16 * 16) : (live + 15) / 16 * 16;
        if (ring_rows > 0) {
            if (!sync()) return false;  // what was there has been read
            if (speaker) {
                const int bytes = (end - begin) * 512;
                asm volatile("fence.proxy.async;" ::: "memory");
                expect_bytes(smem_u32(&s.parts), others * bytes);
                uint32_t to = smem_u32(ring);
                for (int c = first; c <= last; ++c)
                    if (c != cta) bulk_copy(to, slot(c) + begin * 32, bytes, smem_u32(&s.parts)), to += bytes;
            }
            __syncwarp();
            if (!mbar_wait_warp(&s.parts, parts++ & 1, &s.abort, status)) {
                if (speaker) land(&s.parts, (int)parts, 1);
                return false;
            }
        }
#pragma unroll 1
        for (int c0 = begin + 16 * unit0; c0 < end; c0 += 16 * stride) {
            uint32_t v[16];
            tmem_ld16(acc + c0, v);
            tmem_ld_wait();
            if (others > 0) {
                float4 sum[4] = {};
                const float4* h = reinterpret_cast<const float4*>(ring) + (c0 - begin) * 32 + 32 * q + lane;
                for (int c = first; c <= last; ++c) {
                    float4 o[4];
                    if (c == cta) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                                               __uint_as_float(v[4 * i + 3]));
                    } else if (ring_rows > 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[i] = h[i * 128];
                        h += (end - begin) * 32;
                    } else {
                        const float4* const g = slot(c) + c0 * 32 + 32 * q + lane;
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[i] = __ldcg(g + i * 128);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i].x += o[i].x, sum[i].y += o[i].y, sum[i].z += o[i].z, sum[i].w += o[i].w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[4 * i] = __float_as_uint(sum[i].x), v[4 * i + 1] = __float_as_uint(sum[i].y);
                    v[4 * i + 2] = __float_as_uint(sum[i].z), v[4 * i + 3] = __float_as_uint(sum[i].w);
                }
            }
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 g = *reinterpret_cast<const float4*>(sx + c0 + i);
                f[i] = __uint_as_float(v[i]) * g.x * sw;
                f[i + 1] = __uint_as_float(v[i + 1]) * g.y * sw;
                f[i + 2] = __uint_as_float(v[i + 2]) * g.z * sw;
                f[i + 3] = __uint_as_float(v[i + 3]) * g.w * sw;
            }
            T* const y = out + (int64_t)c0 * a.ldy;
            const bool all = whole && c0 + 16 <= live;  // (of the warp)
            if (GATED || pairs) {
                // lanes 2 i and 2 i + 1 exchange: the even one gets both weight rows of row i, the odd one of row i + 1
                float lo[8], hi[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? f[2 * i] : f[2 * i + 1], 1);
                    lo[i] = odd ? got : f[2 * i], hi[i] = odd ? f[2 * i + 1] : got;
                }
                if constexpr (GATED) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) lo[i] = int8_gated(lo[i], hi[i]);
                    if (all) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[2 * i * a.ldy] = int8_result<T>(lo[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (c0 + 2 * i + odd < live && n < N) y[2 * i * a.ldy] = int8_result<T>(lo[i]);
                    }
                } else if (all) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const T u[2] = {int8_result<T>(lo[i]), int8_result<T>(hi[i])};
                        if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(y + 2 * i * a.ldy) = *reinterpret_cast<const uint32_t*>(u);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (c0 + 2 * i + odd < live && (n & ~1) < N) y[2 * i * a.ldy] = int8_result<T>(lo[i]);
                        if (c0 + 2 * i + odd < live && (n | 1) < N) y[2 * i * a.ldy + 1] = int8_result<T>(hi[i]);
                    }
                }
            } else if (all) {
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i * a.ldy] = int8_result<T>(f[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c0 + i < live && n < N) y[i * a.ldy] = int8_result<T>(f[i]);
            }
        }
    }
    return true;
}

template <typename T, bool GATED, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) int8_mma_kernel(const __grid_constant__ MmaArgs args) {
    const Int8ProductArgs& a = args.p;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared& s = *reinterpret_cast<Shared*>(ring + ring_bytes(args));
    unsigned char* const x_ring = ring + args.w_steps * kStepBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_rank() : 0, cta = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x;
    const int KT = (int)((a.K + 63) / 64), KS = (KT + 1) / 2;
    const int NT128 = (int)((a.N + 127) / 128), NT = PAIR ? (NT128 + 1) / 2 : NT128;
    const Work<PAIR> work(s, args);

    if (warp == kWeightWarp) {
        if (lane < kMostStages) {
            mbar_init(&s.w_full[lane], 1);
            mbar_init(&s.w_empty[lane], 8);
            mbar_init(&s.x_full[lane], 1);
            mbar_init(&s.x_empty[lane], 1);
            mbar_init(&s.ready[lane], PAIR ? 17 : 8);
        }
        if (lane < 2) {
            mbar_init(&s.acc_full[lane], 1);
            mbar_init(&s.acc_empty[lane], PAIR ? 2 * kEpiWarps : kEpiWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        mbar_init(&s.epilogue, kEpiWarps);
        mbar_init(&s.all, kFinishWarps);
        mbar_init(&s.parts, 1);
        mbar_init(&s.done, 1);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "r"(kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "r"(kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    if (!a.early) pdl_wait();
    if (warp == 0) {  // the table of the experts' tiles
        int sum = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            int64_t first = 0, count = 0;
            if (e < a.E) {
                first = a.offsets ? int8_offset(a, e) : 0;
                count = a.offsets ? max(int8_offset(a, e + 1) - first, (int64_t)0) : a.M;
            }
            const int own = rows_of(count, args.most).mt * NT;
            int incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (e < a.E) {
                s.tiles[e] = sum + incl - own;
                s.offset[e] = (int32_t)first;
                if (e == a.E - 1) s.offset[a.E] = (int32_t)(first + (a.offsets ? count : 0));
            }
            sum += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            const int G = work.G, rest = sum % G, ctas = min(G, max(rest, (int)min((int64_t)G, (int64_t)rest * KS / kLeastSteps)));
            const bool split = rest > 0 && KS - (int)(((int64_t)rest * KS + ctas - 1) / ctas) >= kLeastSteps;
            s.tiles[a.E] = sum;
            s.split = split ? rest : 0;
            s.ctas = split ? ctas : 0;
            s.whole = sum - s.split;
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // both CTAs' barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    int* const status = &a.ctrl->status;

    if (warp == kWeightWarp) {
        if (elect_one()) {
            Turn t(args.w_steps);
            int it = 0;
            work.each(cta, [&](const Part& p) {
                const int nt = min(PAIR ? 2 * p.nt + rank : p.nt, NT128 - 1);
                const uint8_t* w = a.w + (((int64_t)p.e * NT128 + nt) * KT + 2 * p.k) * kInt8Tile;
                for (int k = p.k; k < p.k1; ++k, w += kStepBytes, ++it, t.next()) {
                    if (!mbar_wait(&s.w_empty[t.at], t.parity ^ 1, &s.abort, status)) return false;
                    const uint32_t bar = smem_u32(&s.w_full[t.at]), bytes = min(2, KT - 2 * k) * kInt8Tile;
                    expect_bytes(bar, bytes);
                    bulk_copy(smem_u32(ring) + t.at * kStepBytes, w, bytes, bar);
                }
                return true;
            });
            land(s.w_full, it, args.w_steps);
        }
    } else if (warp == kRowWarp) {
        if (elect_one()) {
            if (a.early) pdl_wait();
            const int64_t x_step = a.room * 128;
            Turn t(args.x_steps);
            int it = 0;
            work.each(cta, [&](const Part& p) {
                const int n = tile_rows(p) / (PAIR ? 2 : 1), bytes = n * 128;
                const int64_t row = (a.offsets ? int8_first_row(s.offset[p.e], p.e) : 0) + (int64_t)p.mt * p.r.n + (PAIR ? rank * n : 0);
                const uint8_t* x = reinterpret_cast<const uint8_t*>(a.x) + 2 * p.k * x_step + row * 128;
                for (int k = p.k; k < p.k1; ++k, x += 2 * x_step, ++it, t.next()) {
                    if (!mbar_wait(&s.x_empty[t.at], t.parity ^ 1, &s.abort, status)) return false;
                    const uint32_t bar = smem_u32(&s.x_full[t.at]), to = smem_u32(x_ring) + t.at * 2 * args.x_bytes;
                    const bool two = 2 * k + 1 < KT;
                    expect_bytes(bar, two ? 2 * bytes : bytes);
                    bulk_copy(to, x, bytes, bar);
                    if (two) bulk_copy(to + args.x_bytes, x + x_step, bytes, bar);
                }
                return true;
            });
            land(s.x_full, it, args.x_steps);
        }
    } else if (warp == kMmaWarp) {
        if (PAIR && rank != 0) {
            if (elect_one()) {
                Turn t(args.x_steps);
                work.each(cta, [&](const Part& p) {
                    for (int k = p.k; k < p.k1; ++k, t.next()) {
                        if (!mbar_wait(&s.x_full[t.at], t.parity, &s.abort, status)) return false;
                        arrive<PAIR>(&s.ready[t.at]);
                    }
                    return true;
                });
            }
        } else if (elect_one()) {
            const uint32_t base = smem_u32(x_ring);
            Turn t(args.x_steps);
            int tile = 0;
            uint32_t slot = tmem + kSlotBase;
            work.each(cta, [&](const Part& p) {
                const int n = tile_rows(p), b = tile & 1;
                const uint32_t idesc = idesc_f16(PAIR ? 256 : 128, n);
                const uint32_t acc = tmem + b * kMostRows;
                if (!mbar_wait(&s.acc_empty[b], ((tile >> 1) & 1) ^ 1, &s.abort, status)) return false;
                tc_fence_after();
                for (int k = p.k; k < p.k1; ++k, t.next(), slot ^= 2 * kSlotCols) {
                    if (!mbar_wait(&s.x_full[t.at], t.parity, &s.abort, status)) return false;
                    if (!mbar_wait(&s.ready[t.at], t.parity, &s.abort, status)) return false;
                    tc_fence_after();
                    const uint32_t x = ((base + t.at * 2 * args.x_bytes) >> 4) | (1u << 16);
                    step_products<PAIR>(acc, slot, x, idesc, k > p.k ? 1u : 0u);
                    if (2 * k + 1 < KT) step_products<PAIR>(acc, slot + kSlotCols, x + (args.x_bytes >> 4), idesc, 1u);
                    commit<PAIR>(&s.x_empty[t.at]);
                }
                commit<PAIR>(&s.acc_full[b]);
                ++tile;
                return true;
            });
            commit<PAIR>(&s.done);
        }
    } else if (warp < kConvWarps) {
        const int set = warp >> 2, q = warp & 3;
        const unsigned char* w0 = ring + (set & 1) * kInt8Tile + (32 * q + lane) * 16;
        const uint32_t slot = tmem + ((uint32_t)(32 * q) << 16) + kSlotBase + set * kSlotCols;
        // places in the rings: of the step's weights and activations, and of the activations of the step before the last
        Turn t(args.w_steps), x(args.x_steps), old(args.x_steps);
        int it = 0;
        work.each(cta, [&](const Part& p) {
            for (int k = p.k; k < p.k1; ++k, ++it, t.next(), x.next()) {
                if (it >= 3) old.next();
                if ((it & 1) != set >> 1) continue;
                // (The ring has an even number of steps, so that a set waits for every phase of its own places, and not for others': 649 us
                // instead of 676 for the gate and up products of 256 tokens by 8 of 128 experts.)
                if (!mbar_wait_warp(&s.w_full[t.at], t.parity, &s.abort, status)) return false;
                const bool there = 2 * k + (set & 1) < KT;
                uint32_t h[32];
                if (there) convert_row(w0 + t.at * kStepBytes, h);
                // The products of the step before the last have read this slot.  (The phase is not mistaken: this ring is of an even number of
                // steps too, so this set has waited for that of the step which had the same place before.)
                if (it >= 2 && !mbar_wait_warp(&s.x_empty[old.at], old.parity, &s.abort, status)) return false;
                if (there) {
                    tc_fence_after();
                    tmem_st32(slot, h);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.w_empty[t.at]), arrive<PAIR>(&s.ready[x.at]);
            }
            return true;
        });
    } else {
        if (a.early) pdl_wait();
        pdl_launch_dependents();
        uint32_t turn = 0;
        auto sync = [&] {  // of the epilogue's warps; bounded, like every wait
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.epilogue);
            return mbar_wait_warp(&s.epilogue, turn++ & 1, &s.abort, status);
        };
        int tile = 0;
        work.each(cta, [&](const Part& p) {
            if (p.last) return false;
            if (!finish<T, GATED, PAIR>(args, s, ring, work, tmem, p, tile, 0, 1, s.sx[warp & 3], &s.last[tile & 1], sync)) return false;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive<PAIR>(&s.acc_empty[tile & 1]);
            ++tile;
            return true;
        });
    }
    // The CTA's last part is finished by the converting warps too, which have nothing else to do then: five warps a lane quarter.
    if (warp < kFinishWarps) {
        __syncwarp();
        // (Everything it needs is found again from here: what lives on until here costs the loops above registers.)
        const MmaArgs* args2 = &args;
        unsigned char* raw2 = smem_raw;
        asm volatile("" : "+l"(args2), "+l"(raw2));
        unsigned char* const ring2 = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw2) + 1023) & ~uintptr_t(1023));
        Shared& s2 = *reinterpret_cast<Shared*>(ring2 + ring_bytes(*args2));
        const Work<PAIR> work2(s2, *args2);
        Part p;
        const int tile = work2.last(PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x, p), part = (int)threadIdx.x >> 7;
        if (tile >= 0 && !s2.abort) {
            if (args2->p.early && part < kSets) pdl_wait();
            uint32_t turn = 0;
            auto sync = [&] {
                __syncwarp();
                if (threadIdx.x % 32 == 0) mbar_arrive(&s2.all);
                return mbar_wait_warp(&s2.all, turn++ & 1, &s2.abort, &args2->p.ctrl->status);
            };
            // (the epilogue's warps, which have been waiting for the accumulators, take the first rows)
            finish<T, GATED, PAIR>(*args2, s2, ring2, work2, s2.tmem, p, tile, (part + 1) % (kFinishWarps / 4), kFinishWarps / 4, s2.sx[4], &s2.last[2],
                                   sync);
            tc_fence_before();
        }
    }
    __syncwarp();
    {
        // every product has completed: the leader commits `done` last, aborting or not
        volatile int never = 0;
        mbar_wait(&s.done, 0, &never, nullptr);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // neither CTA's shared or tensor memory goes while the other may use it
    if (warp == kMmaWarp) {
        tc_fence_after();
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <typename T, bool GATED>
const void* mma_kernel(bool pair) {
    return pair ? (const void*)int8_mma_kernel<T, GATED, true> : (const void*)int8_mma_kernel<T, GATED, false>;
}
template <typename T>
const void* mma_kernel(bool gated, bool pair) {
    return gated ? mma_kernel<T, true>(pair) : mma_kernel<T, false>(pair);
}

}  // namespace

cudaError_t launch_int8_mma(const Int8ProductArgs& a, moe_dtype dtype, bool gated, bool pair, cudaStream_t st) {
    MmaArgs m = {};
    m.p = a;
    m.slot_rows = (int)(a.M > kMostRows ? kMostRows : (a.M + 15) / 16 * 16);
    // By expert the ring has room for tiles of four times the mean, or 64 rows above it (more of an expert's rows are several tiles): small
    // ones leave room for more steps of weights on their way.
    const int64_t mean = a.M / a.E, cap = mean + (mean < 16 ? 3 * mean + 16 : 64), rows = a.offsets && cap < a.M ? cap : a.M;
    m.most = (int)(rows > kMostRows ? kMostRows : (rows + 15) / 16 * 16);
    m.x_bytes = m.most * 128 / (pair ? 2 : 1);
    m.x_bytes = (m.x_bytes + 1023) / 1024 * 1024;
    // At least 4 steps of activations (3: 185 us instead of 155 for 4096 x 4096 x 8192), or 6 where these leave 6 of weights; as many of
    // weights as that leaves, and what these leave.
    const int fit = (int)(kSmemMost - 1024 - sizeof(Shared)) / 1024 * 1024, x_step = 2 * m.x_bytes;
    m.w_steps = (fit - (fit - 6 * x_step >= 6 * kStepBytes ? 6 : 4) * x_step) / kStepBytes / 2 * 2;
    if (m.w_steps > kMostStages) m.w_steps = kMostStages;
    m.x_steps = (fit - m.w_steps * kStepBytes) / x_step / 2 * 2;
    if (m.x_steps > kMostStages) m.x_steps = kMostStages;
    // (more than half of the SM's shared memory, so that one CTA per SM owns its tensor memory)
    size_t smem = (size_t)ring_bytes(m) + sizeof(Shared) + 1024;
    if (smem < 120 * 1024) smem = 120 * 1024;
    int ctas = sm_count() < kInt8Ctas ? sm_count() : kInt8Ctas;
    if (pair) ctas = ctas / 2 * 2;
    const void* f = dtype == MOE_F32    ? mma_kernel<float>(gated, pair)
                    : dtype == MOE_BF16 ? mma_kernel<__nv_bfloat16>(gated, pair)
                                        : mma_kernel<__half>(gated, pair);
    void* args[] = {&m};
    return launch_cluster(f, dim3(ctas), kThreads, smem, pair ? 2 : 1, st, args);
}

}  // namespace moe
