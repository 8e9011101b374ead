// nvfp4_operand.cu -- NVFP4 operands of the dense product: E2M1 codes, one E4M3 scale per 16 elements along
// the contraction and one fp32 scale per operand row, written straight in the tensor-core layout, from a
// matrix x [R][C] of fp32, bf16 or fp16 (row stride ld), its transpose, or both.
//
// The rule is the weight packer's, row by row: g = max|row| / 2688 (1 when 0); per block t = (max|block| / g) / 6,
// scale = nearest E4M3 (ties to even, saturating), D = scale * g, code = nearest E2M1 to v / D; every step
// in fp32, rounded to nearest even.  A row's own scale keeps a token's operand independent of the other
// tokens of its batch.
//
// Quotients cost three fp32 operations each: q0 = a y, q = q0 + (a - q0 b) y with y = 1 / b rounded (Markstein's
// correction, IBM J. Res. Dev. 34, 1990).  Checked exhaustively on a CPU: for v / D, over all 2^23 mantissas of D and all
// v within six ulps of the seven values where the code changes, q decides as the rounded quotient does
// (without the correction 4% of those decisions differ, and farther away one ulp cannot change a code);
// for max|block| / g with a 16-bit numerator and for t / 6, q is the rounded quotient.  1 / D itself is the hardware's
// reciprocal with one Newton step; a GPU test runs all mantissas of D against the division.  fp32 maxima, and
// row scales outside 2^-50 .. 2^50, take the division.
//
// A thread encodes blocks of 16: their maximum is taken on the packed bits (two 16-bit elements per instruction).
//   rows only   the threads of a row hold it in registers (up to 8192 elements), reduce its maximum, encode; many rows
//               are streamed through shared memory by persistent CTAs.
//   with columns  two passes over x: the row and column maxima (integer maxima of the bits: the order of the
//               atomics does not matter), then tiles of 256 rows x 64 columns through shared memory, encoded
//               along their rows and along their columns, two columns per thread; 256 rows are a whole
//               128-byte row of a column operand's code tile.  The second pass finds x in L2 while it fits there.
// (2 or 4) R C bytes in, 9/16 R C out per form.  Rows of a bf16 matrix 4096 x 8192: 18 us (4.8 TB/s), both forms 44.6 us (11 of
// them the maxima).  The encoding, about 110 warp instructions per block and lane, keeps 58% of the issue slots busy; leaving out
// the stores (43.7 us) or smaller tiles with a third more warps (49) hardly matter or hurt.
#include <type_traits>

#include "ops.cuh"
#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTileR = 256, kTileC = 64;  // rows and columns of a tile of the two-form kernel

__host__ __device__ inline int64_t pad_to(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// 16 consecutive elements as they are in memory.
template <typename T>
struct Block {
    static constexpr int kWords = 4 * (int)sizeof(T);
    uint32_t w[kWords];

    __device__ __forceinline__ void load_wide(const T* p) {  // p is 16-byte aligned
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
    // those at or past `live` are zero
    __device__ __forceinline__ void load(const T* p, int64_t live, bool wide) {
        if (wide && live >= 16) {
            load_wide(p);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = i < live ? __float_as_uint(p[i]) : 0u;
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = (2 * i < live ? (uint32_t)h[2 * i] : 0u) | (2 * i + 1 < live ? (uint32_t)h[2 * i + 1] << 16 : 0u);
        }
    }
    __device__ __forceinline__ void values(float (&v)[16]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    const float2 f = h2_to_f2(w[i]);
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            }
        }
    }
};

// The first `bytes` (0 .. 16) of 16 bytes; zeros after them.
__device__ __forceinline__ void cp_async16_part(void* smem, const void* gmem, int bytes) {
    const uint32_t sa = (uint32_t)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sa), "l"(gmem), "r"(bytes) : "memory");
}

// The same of 4 bytes.
__device__ __forceinline__ void cp_async4_part(void* smem, const void* gmem, int bytes) {
    const uint32_t sa = (uint32_t)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sa), "l"(gmem), "r"(bytes) : "memory");
}
// Shared memory of a warp's 32 units in the streaming kernel.
template <typename T, bool WIDE>
__host__ __device__ constexpr int stream_warp_bytes() { return WIDE ? 32 * 32 * (int)sizeof(T) : (32 * (8 * (int)sizeof(T) + 1) + 4) * 4; }

// The larger magnitudes of a word of one fp32 or two 16-bit elements (a: magnitudes already).  A NaN is the largest of all, so that it
// reaches the scale: as an integer of fp32 bits it is by itself.
template <typename T>
__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) {
        return max(a, b & 0x7fffffffu);
    } else {
        uint32_t r;
        if constexpr (std::is_same<T, __half>::value) {
            asm("{\n\t.reg .b32 m;\n\tabs.f16x2 m, %2;\n\tmax.NaN.f16x2 %0, %1, m;\n\t}" : "=r"(r) : "r"(a), "r"(b));
        } else {
            asm("{\n\t.reg .b32 m;\n\tabs.bf16x2 m, %2;\n\tmax.NaN.bf16x2 %0, %1, m;\n\t}" : "=r"(r) : "r"(a), "r"(b));
        }
        return r;
    }
}
// A maximum of magnitudes as fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t mag_f32(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return max(m << 16, m & 0xffff0000u);
    else {
        const float2 f = h2_to_f2(m);
        return max(__float_as_uint(f.x), __float_as_uint(f.y));
    }
}
template <typename T>
__device__ __forceinline__ uint32_t block_mag(const Block<T>& b) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < Block<T>::kWords; ++i) m = mag_max<T>(m, b.w[i]);
    return mag_f32<T>(m);
}

__device__ __forceinline__ float quotient(float a, float b, float y) {  // y = 1 / b rounded
    const float q0 = __fmul_rn(a, y);
    return __fmaf_rn(__fmaf_rn(-q0, b, a), y, q0);
}

// A row scale and its reciprocal (0: outside 2^-50 .. 2^50, where quotients take the division).  A block scale of at
// least 2^-9 and at most 448 keeps D = scale * g inside the range where no step of a quotient loses bits.
struct RowScale {
    float g, y;
};
__device__ __forceinline__ RowScale with_reciprocal(float g) {
    return {g, g >= 8.8817842e-16f && g <= 1.1258999e15f ? __frcp_rn(g) : 0.f};
}
// That of a row's largest magnitude: max / 2688, or 1 (the quotient is the rounded one for every mantissa).
__device__ __forceinline__ RowScale row_scale(uint32_t mag) {
    const float m = __uint_as_float(mag);
    float g = quotient(m, 2688.f, 1.f / 2688.f);
    if (!(m >= 1e-12f && m <= 1e18f)) {
        g = __fdiv_rn(m, 2688.f);
        if (g == 0.f) g = 1.f;
    }
    return with_reciprocal(g);
}

// One block of 16 elements of largest magnitude amax under the row scale: 8 bytes of codes; returns the scale byte.
// PLAIN: rs.y is not 0 and the scale is the row's own; given: it may not be, and quotients may be far above 6: they saturate.  The block's
// scale is then found by divisions, which give inf and not NaN where they overflow, and by a scale of zero as by the smallest
// number: its blocks of zeros stay zeros (0 / 0 would make them NaN), and D = 0 makes zeros of all others.
template <typename T, bool PLAIN>
__device__ __forceinline__ uint32_t encode_block(float (&v)[16], float amax, RowScale rs, bool given, uint2& codes) {
    float t;
    if (sizeof(T) == 2 && PLAIN) t = quotient(quotient(amax, rs.g, rs.y), 6.f, 0.166666672f);
    else t = __fdiv_rn(__fdiv_rn(amax, PLAIN ? rs.g : fmaxf(rs.g, 1e-45f)), 6.f);
    const uint32_t sb = f32_to_e4m3_sat(t);
    const float D = __fmul_rn(e4m3x2_to_f2(sb).x, rs.g);
    if (!PLAIN && given) {
        const float lim = 8.f * D;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = fminf(fmaxf(v[i], -lim), lim);
    }
    if (PLAIN || rs.y != 0.f) {
        float y;  // 1 / D rounded (the hardware's reciprocal and a Newton step); a zero scale gives zero codes
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(D));
        y = sb == 0 ? 0.f : fmaf(y, fmaf(-D, y, 1.f), y);
        const float2 y2 = make_float2(y, y), d2 = make_float2(-D, -D);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {  // quotient() on pairs (q0 = a y + (-0): the rounded product)
            const float2 a = make_float2(v[i], v[i + 1]);
            const float2 q0 = fma2(a, y2, make_float2(-0.f, -0.f));
            const float2 q = fma2(fma2(q0, d2, a), y2, q0);
            v[i] = q.x;
            v[i + 1] = q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = D == 0.f ? 0.f : __fdiv_rn(v[i], D);
    }
    codes = make_uint2(e2m1x8_encode(v), e2m1x8_encode(v + 8));
    return sb;
}

// Byte offsets inside a 128-row block of an operand of width Kp: of the 16 bytes of codes of unit u (32
// elements: two blocks) of row `in`, and of its two scales.
__device__ __forceinline__ uint32_t unit_codes(uint32_t in, uint32_t u) {
    return (u >> 3) * 16384u + in * 128u + (((u & 7u) ^ (in & 7u)) * 16u);
}
__device__ __forceinline__ uint32_t unit_scales(uint32_t in, uint32_t u) {
    return (u >> 1) * 512u + (in & 31u) * 16u + (in >> 5) * 4u + 2u * (u & 1u);
}

// Two adjacent blocks of a row: 16 bytes of codes; the lanes of two adjacent units (u even in the even lane) store their
// four scales as one word.
template <typename T>
__device__ __forceinline__ void encode_unit(const Block<T>& a, const Block<T>& b, uint32_t mag_a, uint32_t mag_b, RowScale rs, bool given,
                                            uint8_t* q, uint8_t* s, bool live) {
    float v[16];
    uint2 ca, cb;
    uint32_t word;
    if (!given && rs.y != 0.f) {
        a.values(v);
        word = encode_block<T, true>(v, __uint_as_float(mag_a), rs, false, ca);
        b.values(v);
        word |= encode_block<T, true>(v, __uint_as_float(mag_b), rs, false, cb) << 8;
    } else {
        a.values(v);
        word = encode_block<T, false>(v, __uint_as_float(mag_a), rs, given, ca);
        b.values(v);
        word |= encode_block<T, false>(v, __uint_as_float(mag_b), rs, given, cb) << 8;
    }
    if (live) *reinterpret_cast<uint4*>(q) = make_uint4(ca.x, ca.y, cb.x, cb.y);
    word |= __shfl_down_sync(0xffffffffu, word, 1) << 16;
    if (live && (threadIdx.x & 1) == 0) *reinterpret_cast<uint32_t*>(s) = word;
}

// ------------------------------------------------------------------ rows only
// tpr = 2^tpr_log threads (32 .. 256) share a row; thread c of them the units (two blocks) c, c + tpr, ...; the
// first stays in registers.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
    nvfp4_rows_kernel(const T* __restrict__ x, int64_t R, int64_t K, int64_t ld, bool wide, int tpr_log, uint8_t* __restrict__ q,
                      uint8_t* __restrict__ s, float* __restrict__ gs, bool given, bool gs_rows) {
    __shared__ __align__(16) uint32_t part[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();  // a product launched behind this call fetches its weights meanwhile
    const int tpr = 1 << tpr_log, u0 = threadIdx.x & (tpr - 1);
    const int64_t first = (int64_t)blockIdx.x * (kThreads >> tpr_log);  // the CTA's rows: inside one 128-row block
    const uint32_t sub = threadIdx.x >> tpr_log;
    const bool live = first + sub < R;
    const int units = (int)((K + 255) >> 8) * 8;
    const int whole = wide ? (int)(K >> 5) : 0;  // units that are read in 16-byte pieces
    const T* row = x + first * ld + (live ? sub * ld : 0);
    Block<T> a, b;
    auto load = [&](int u) {
        const T* p = row + 32 * (int64_t)u;
        if (u < whole) {
            a.load_wide(p);
            b.load_wide(p + 16);
        } else {
            const int64_t left = u < units ? K - 32 * (int64_t)u : 0;
            a.load(p, left, wide);
            b.load(p + 16, left - 16, wide);
        }
    };
    load(u0);
    uint32_t mag_a = block_mag(a), mag_b = block_mag(b);
    RowScale rs = {1.f, 0.f};
    if (!given) {
        uint32_t m = max(mag_a, mag_b);
        if (units > tpr) {
#pragma unroll 1
            for (int u = u0 + tpr; u < units; u += tpr) {
                load(u);
                m = max(m, max(block_mag(a), block_mag(b)));
            }
            load(u0);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (tpr > 32) {
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
            __syncthreads();
            const int w0 = (threadIdx.x >> tpr_log) << (tpr_log - 5);
            if (tpr == kThreads) {
                const uint4 lo = *reinterpret_cast<const uint4*>(part), hi = *reinterpret_cast<const uint4*>(part + 4);
                m = max(max(max(lo.x, lo.y), max(lo.z, lo.w)), max(max(hi.x, hi.y), max(hi.z, hi.w)));
            } else {
                for (int w = 0; w < tpr >> 5; ++w) m = max(m, part[w0 + w]);
            }
        }
        rs = row_scale(m);
        if (live && u0 == 0) gs[first + sub] = rs.g;
    } else if (live) {
        rs = with_reciprocal(gs[gs_rows ? first + sub : 0]);
    }
    const uint32_t in = ((uint32_t)first & 127u) + sub;  // row of its 128-row block
    q += (first >> 7) * units * 2048;
    s += (first >> 7) * units * 256;
    int64_t at = unit_codes(in, u0), sat = unit_scales(in, u0);
    int u = u0;
    while (true) {
        encode_unit(a, b, mag_a, mag_b, rs, given, q + at, s + sat, live && u < units);
        u += tpr;
        if (u - u0 >= units) break;  // (all threads of a row together)
        at += tpr * 2048, sat += tpr * 256;
        load(u);
        mag_a = block_mag(a), mag_b = block_mag(b);
    }
}

// Rows of up to 8192 elements: persistent CTAs, each with the next row's copy (cp.async) in flight while this one is reduced and
// encoded.  A warp reads and encodes what it copied itself.
//   WIDE   rows that start on 16 bytes, where there are more than twice what the SMs hold at once: pieces of 16 bytes, swizzled, so that
//          lanes reading a unit each meet all banks.
//   else   words of 4 bytes from the aligned one that holds the row's first element (its other half, when the element is the
//          second of two, lies in front of it in the same allocation, which starts on 4 bytes at least), a word of padding per
//          unit; a row that starts on 2 bytes is shifted while it is read.  4096 x 8191 bf16: 24.6 us, 64 where every thread
//          loads its own elements.
template <typename T, int CTAS, bool WIDE>
__global__ void __launch_bounds__(kThreads, CTAS)
    nvfp4_rows_stream_kernel(const T* __restrict__ x, int64_t R, int64_t K, int64_t ld, int tpr_log, uint8_t* __restrict__ q,
                             uint8_t* __restrict__ s, float* __restrict__ gs, bool given, bool gs_rows) {
    extern __shared__ __align__(16) unsigned char rows_smem[];  // two buffers of 32 elements per thread
    __shared__ __align__(16) uint32_t part[2][kThreads / 32];
    constexpr int kPieces = 32 * (int)sizeof(T) / 16, kPer = 16 / (int)sizeof(T), kUnitWords = 4 * kPieces;
    constexpr int kWarpBytes = stream_warp_bytes<T, WIDE>(), kBuffer = kThreads / 32 * kWarpBytes;
    pdl_wait();
    pdl_launch_dependents();
    const int tpr = 1 << tpr_log, rpc = kThreads >> tpr_log;  // threads a row, rows a turn
    const int u0 = threadIdx.x & (tpr - 1), lane = threadIdx.x & 31;
    const uint32_t sub = threadIdx.x >> tpr_log;
    const int units = (int)((K + 255) >> 8) * 8;
    const int64_t turns = (R + rpc - 1) / rpc;
    unsigned char* mine = rows_smem + (threadIdx.x >> 5) * kWarpBytes;  // this warp's pieces
    const int warp_e = (u0 & ~31) * 32;  // first element of the warp's part of its row
    auto fetch = [&](int64_t turn, unsigned char* to) {
        const int64_t r = turn * rpc + sub;
        const T* row = x + (r < R ? r : R - 1) * ld;
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = 32 * i + lane, e = warp_e + p * kPer;
                const int64_t left = (K - e) * (int64_t)sizeof(T);
                cp_async16_part(to + (p ^ ((p >> 3) & 7)) * 16, row + (left > 0 ? e : 0), left >= 16 ? 16 : left > 0 ? (int)left : 0);
            }
        } else {
            const int ahead = sizeof(T) == 2 ? (int)(reinterpret_cast<uintptr_t>(row) & 2) : 0;
            const char* first = reinterpret_cast<const char*>(row) - ahead;
            const char* from = first + warp_e * (int)sizeof(T) + 4 * lane;
            unsigned char* at = to + 4 * (lane + lane / kUnitWords);
            // bytes of the row from this lane's first word on
            const int64_t left = (K - warp_e) * (int64_t)sizeof(T) + ahead - 4 * lane;
            constexpr int kTurn = 4 * (32 + 32 / kUnitWords);
            if ((K - warp_e) * (int64_t)sizeof(T) >= 128 * kUnitWords) {
#pragma unroll
                for (int i = 0; i < kUnitWords; ++i) cp_async4_part(at + kTurn * i, from + 128 * i, 4);
            } else {
#pragma unroll 4
                for (int i = 0; i < kUnitWords; ++i) {
                    const int n = (int)max((int64_t)0, min((int64_t)4, left - 128 * i));
                    cp_async4_part(at + kTurn * i, n > 0 ? from + 128 * i : first, n);
                }
            }
            if (sizeof(T) == 2 && lane == 0) {  // the word that the last lane's unit ends in
                const int n = (int)max((int64_t)0, min((int64_t)4, left - 128 * kUnitWords));
                cp_async4_part(at + kTurn * kUnitWords, n > 0 ? from + 128 * kUnitWords : first, n);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](Block<T>& blk, const unsigned char* from, int h, int ahead) {  // block h of this lane's unit
        if constexpr (WIDE) {
#pragma unroll
            for (int j = 0; j < kPieces / 2; ++j) {
                const int p = lane * kPieces + h * (kPieces / 2) + j;
                const uint4 v = *reinterpret_cast<const uint4*>(from + (p ^ ((p >> 3) & 7)) * 16);
                blk.w[4 * j] = v.x, blk.w[4 * j + 1] = v.y, blk.w[4 * j + 2] = v.z, blk.w[4 * j + 3] = v.w;
            }
        } else {
            constexpr int kHalf = kUnitWords / 2;
            const uint32_t* word = reinterpret_cast<const uint32_t*>(from) + (kUnitWords + 1) * lane + kHalf * h;
#pragma unroll
            for (int j = 0; j < kHalf; ++j) blk.w[j] = word[j];
            if (ahead) {  // (after a unit's last word comes its padding)
                const uint32_t next = word[h == 0 ? kHalf : kHalf + 1];
#pragma unroll
                for (int j = 0; j < kHalf; ++j) blk.w[j] = __funnelshift_r(blk.w[j], j + 1 < kHalf ? blk.w[j + 1] : next, 16);
            }
        }
    };
    fetch(blockIdx.x, mine);
    int buf = 0;
    for (int64_t turn = blockIdx.x; turn < turns; turn += gridDim.x, buf ^= 1) {
        if (turn + gridDim.x < turns) {
            fetch(turn + gridDim.x, mine + (buf ^ 1) * kBuffer);
            cp_async_wait_group<1>();
        } else {
            cp_async_wait_group<0>();
        }
        __syncwarp();
        const int64_t r = turn * rpc + sub;
        const bool live = r < R;
        Block<T> a, b;
        const int ahead = !WIDE && sizeof(T) == 2 ? (int)(reinterpret_cast<uintptr_t>(x + (live ? r : R - 1) * ld) & 2) : 0;
        take(a, mine + buf * kBuffer, 0, ahead);
        take(b, mine + buf * kBuffer, 1, ahead);
        const uint32_t mag_a = block_mag(a), mag_b = block_mag(b);
        RowScale rs = {1.f, 0.f};
        if (!given) {
            uint32_t m = __reduce_max_sync(0xffffffffu, max(mag_a, mag_b));
            if (tpr > 32) {
                if (lane == 0) part[buf][threadIdx.x >> 5] = m;
                __syncthreads();
                if (tpr == kThreads) {
                    const uint4 lo = *reinterpret_cast<const uint4*>(part[buf]), hi = *reinterpret_cast<const uint4*>(part[buf] + 4);
                    m = max(max(max(lo.x, lo.y), max(lo.z, lo.w)), max(max(hi.x, hi.y), max(hi.z, hi.w)));
                } else {
                    const int w0 = (threadIdx.x >> tpr_log) << (tpr_log - 5);
                    for (int w = 0; w < tpr >> 5; ++w) m = max(m, part[buf][w0 + w]);
                }
            }
            rs = row_scale(m);
            if (live && u0 == 0) gs[r] = rs.g;
        } else if (live) {
            rs = with_reciprocal(gs[gs_rows ? r : 0]);
        }
        const uint32_t in = (uint32_t)r & 127u;
        const int64_t block = (r >> 7) * units;
        encode_unit(a, b, mag_a, mag_b, rs, given, q + block * 2048 + unit_codes(in, u0), s + block * 256 + unit_scales(in, u0),
                    live && u0 < units);
        __syncwarp();  // the buffer is free
    }
}

// ------------------------------------------------------------------ with columns
// 16 bytes of elements from p on, of which `left` are in the row: zeros after them.  p may start anywhere: aligned words, shifted
// (an element in front of p or behind the 16 bytes may be read with them, in words that hold elements of the piece or the row).
template <typename T>
__device__ __forceinline__ uint4 load_piece(const T* p, int64_t left) {
    constexpr int kPer = 16 / (int)sizeof(T);
    const uint32_t ahead = sizeof(T) == 2 ? (uint32_t)(reinterpret_cast<uintptr_t>(p) & 2) : 0u;
    if (left > kPer || (left == kPer && ahead == 0)) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(reinterpret_cast<const char*>(p) - ahead);
        const uint32_t a = __ldg(q), b = __ldg(q + 1), c = __ldg(q + 2), d = __ldg(q + 3), e = ahead ? __ldg(q + 4) : 0u;
        return make_uint4(__funnelshift_r(a, b, 8 * ahead), __funnelshift_r(b, c, 8 * ahead), __funnelshift_r(c, d, 8 * ahead),
                          __funnelshift_r(d, e, 8 * ahead));
    }
    __align__(16) T t[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) t[i] = i < left ? p[i] : T(0.f);
    return *reinterpret_cast<const uint4*>(t);
}

__global__ void __launch_bounds__(kThreads) nvfp4_zero_kernel(unsigned* p, int64_t n) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i < n) p[i] = 0u;
}

// Maxima of |x| over rows and columns as fp32 bits in row_max[R] and col_max[C], which the kernel before zeroes meanwhile: x is
// read ahead of the wait, since that kernel has waited for what was written before it.  A warp takes kMaxRows rows of 16 bytes per lane; the 8 warps of a CTA rows of the same columns.
constexpr int kMaxRows = 16;
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
    nvfp4_maxima_kernel(const T* __restrict__ x, int64_t R, int64_t C, int64_t ld, bool wide, int col_tiles,
                        unsigned* __restrict__ row_max, unsigned* __restrict__ col_max) {
    constexpr int kPer = 16 / (int)sizeof(T), kWarpCols = 32 * kPer;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ uint32_t part[kThreads / 32][kWarpCols];
    pdl_launch_dependents();
    const int64_t col0 = (blockIdx.x % col_tiles) * (int64_t)kWarpCols;
    const int64_t c0 = col0 + kPer * lane, r0 = ((int64_t)(blockIdx.x / col_tiles) * (kThreads / 32) + warp) * kMaxRows;
    uint32_t cm[4] = {0u, 0u, 0u, 0u};
    unsigned mine = 0;
    const int rows = (int)max((int64_t)0, min((int64_t)kMaxRows, R - r0));
    for (int j0 = 0; j0 < rows; j0 += 8) {
        uint4 u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] = make_uint4(0u, 0u, 0u, 0u);
            if (j0 + j >= rows || c0 >= C) continue;
            const T* p = x + (r0 + j0 + j) * ld + c0;
            if (wide && c0 + kPer <= C) {
                u[j] = __ldg(reinterpret_cast<const uint4*>(p));
            } else {
                u[j] = load_piece(p, C - c0);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cm[0] = mag_max<T>(cm[0], u[j].x);
            cm[1] = mag_max<T>(cm[1], u[j].y);
            cm[2] = mag_max<T>(cm[2], u[j].z);
            cm[3] = mag_max<T>(cm[3], u[j].w);
            const uint32_t m = mag_max<T>(mag_max<T>(mag_max<T>(mag_max<T>(0u, u[j].x), u[j].y), u[j].z), u[j].w);
            const unsigned rm = __reduce_max_sync(0xffffffffu, mag_f32<T>(m));
            if (lane == j0 + j) mine = rm;
        }
    }
    pdl_wait();
    if (row_max && lane < rows) atomicMax(row_max + r0 + lane, mine);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            part[warp][kPer * lane + i] = cm[i];
        } else {
            part[warp][kPer * lane + 2 * i] = mag_f32<T>(cm[i] & 0xffffu);
            part[warp][kPer * lane + 2 * i + 1] = mag_f32<T>(cm[i] >> 16);
        }
    }
    __syncthreads();
    if (threadIdx.x >= kWarpCols || col0 + threadIdx.x >= C) return;
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, part[w][threadIdx.x]);
    atomicMax(col_max + col0 + threadIdx.x, m);
}

// Tiles of 256 x 64 elements of x in shared memory, encoded along their rows (a thread: 2 units) and along their
// columns (a thread: 2 columns x 32 rows; eight lanes hold the 256 rows of a column and write its 128 bytes of
// codes).  The 16-byte pieces of a row are rotated by its group of 32 rows, so that lanes reading 8 groups x 4
// words meet all banks.  Tiles cover the padded contractions (256 multiples), whose padding is written as zeros.
// Persistent CTAs: the next tile is fetched (cp.async, a second buffer) while this one is encoded.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 1 : 3)
    nvfp4_both_kernel(const T* __restrict__ x, int64_t R, int64_t C, int64_t ld, bool wide, int col_tiles, int n_tiles,
                      const unsigned* row_max, const unsigned* col_max,
                      const __grid_constant__ moe_nvfp4_operand rows, const __grid_constant__ moe_nvfp4_operand cols, bool given) {
    extern __shared__ __align__(16) unsigned char tiles[];  // two buffers
    __shared__ RowScale row_scales[kTileR], col_scales[kTileC];
    constexpr int kPitch = kTileC * (int)sizeof(T), kPer = 16 / (int)sizeof(T), kPieces = kTileC / kPer, kTurn = kPieces / 8;
    const int64_t Cp = pad_to(C, 256), Rp = pad_to(R, 256);
    auto place = [&](int rr, int pc) { return rr * kPitch + ((pc + kTurn * (rr >> 5)) & (kPieces - 1)) * 16; };
    float row_v = 0.f, col_v = 0.f;  // this thread's row and column scale (or maximum) of the tile to come
    auto fetch = [&](int t, unsigned char* to) {
        const int64_t r0 = (int64_t)(t / col_tiles) * kTileR, c0 = (int64_t)(t % col_tiles) * kTileC;
        if (wide && r0 + kTileR <= R && c0 + kTileC <= C) {
            constexpr int kStep = kThreads / kPieces;  // rows per turn: 32, or 16 of fp32
            const int rr = threadIdx.x / kPieces, pc = threadIdx.x % kPieces;
            const T* p = x + (r0 + rr) * ld + c0 + pc * kPer;
#pragma unroll
            for (int i = 0; i < kTileR / kStep; ++i, p += kStep * ld) cp_async16(to + place(rr + i * kStep, pc), p);
        } else if (wide) {  // at the edges
#pragma unroll 1
            for (int i = threadIdx.x; i < kTileR * kPieces; i += kThreads) {
                const int rr = i / kPieces, pc = i % kPieces;
                const int64_t r = r0 + rr, c = c0 + pc * kPer, left = r < R && c < C ? (C - c) * (int64_t)sizeof(T) : 0;
                cp_async16_part(to + place(rr, pc), left > 0 ? x + r * ld + c : x, left >= 16 ? 16 : (int)left);
            }
        } else {
            constexpr int kFly = 4;  // pieces in flight
            static_assert(kTileR * kPieces % (kFly * kThreads) == 0, "whole turns");
#pragma unroll 1
            for (int i = threadIdx.x; i < kTileR * kPieces; i += kFly * kThreads) {
                uint4 v[kFly];
#pragma unroll
                for (int h = 0; h < kFly; ++h) {
                    const int rr = (i + h * kThreads) / kPieces, pc = (i + h * kThreads) % kPieces;
                    const int64_t r = r0 + rr, c = c0 + pc * kPer;
                    v[h] = r < R ? load_piece(x + r * ld + c, C - c) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int h = 0; h < kFly; ++h)
                    *reinterpret_cast<uint4*>(to + place((i + h * kThreads) / kPieces, (i + h * kThreads) % kPieces)) = v[h];
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto fetch_scales = [&](int t) {
        const int64_t r = (int64_t)(t / col_tiles) * kTileR + threadIdx.x, c = (int64_t)(t % col_tiles) * kTileC + threadIdx.x;
        if (rows.q && r < R) row_v = given ? rows.gs[rows.gs_rows ? r : 0] : __uint_as_float(__ldcg(row_max + r));
        if (threadIdx.x < kTileC && c < C) col_v = given ? cols.gs[cols.gs_rows ? c : 0] : __uint_as_float(__ldcg(col_max + c));
    };
    if (given) pdl_wait();  // else x is there: the kernel before the maxima's has waited for it
    fetch(blockIdx.x, tiles);
    pdl_wait();  // the maxima
    pdl_launch_dependents();
    fetch_scales(blockIdx.x);
    int buf = 0;
    for (int t = blockIdx.x; t < n_tiles; t += gridDim.x, buf ^= 1) {
        const int64_t r0 = (int64_t)(t / col_tiles) * kTileR, c0 = (int64_t)(t % col_tiles) * kTileC;
        unsigned char* tile = tiles + buf * (kTileR * kPitch);
        auto piece_at = [&](int rr, int pc) { return tile + place(rr, pc); };
        if (rows.q) {
            const RowScale rs = given ? with_reciprocal(row_v) : row_scale(__float_as_uint(row_v));
            row_scales[threadIdx.x] = rs;
            if (!given && c0 == 0 && r0 + threadIdx.x < R) rows.gs[r0 + threadIdx.x] = rs.g;
        }
        if (threadIdx.x < kTileC) {
            const RowScale rs = given ? with_reciprocal(col_v) : row_scale(__float_as_uint(col_v));
            col_scales[threadIdx.x] = rs;
            if (!given && r0 == 0 && c0 + threadIdx.x < C) cols.gs[c0 + threadIdx.x] = rs.g;
        }
        if (t + (int)gridDim.x < n_tiles) {
            fetch(t + gridDim.x, tiles + (buf ^ 1) * (kTileR * kPitch));
            fetch_scales(t + gridDim.x);
            cp_async_wait_group<1>();
        } else {
            cp_async_wait_group<0>();
        }
        __syncthreads();
        if (rows.q) {
            // thread: row threadIdx / 2 (+ 128), unit threadIdx % 2 of the tile's 64 columns
            const uint32_t in = threadIdx.x >> 1, u = threadIdx.x & 1;
            const int64_t units = Cp / 32;
            uint8_t* q = rows.q + (r0 >> 7) * units * 2048 + unit_codes(in, (uint32_t)(c0 >> 5) & 7u | u) + (c0 >> 8) * 16384;
            uint8_t* s = rows.s + (r0 >> 7) * units * 256 + unit_scales(in, u) + (c0 >> 6) * 512;
#pragma unroll 1
            for (int i = 0; i < 2; ++i, q += units * 2048, s += units * 256) {
                const int rr = 128 * i + in;
                Block<T> a, b;
                constexpr int kBlockPieces = Block<T>::kWords / 4;
#pragma unroll
                for (int j = 0; j < kBlockPieces; ++j) {
                    const uint4 x0 = *reinterpret_cast<const uint4*>(piece_at(rr, 2 * u * kBlockPieces + j));
                    const uint4 x1 = *reinterpret_cast<const uint4*>(piece_at(rr, (2 * u + 1) * kBlockPieces + j));
                    a.w[4 * j] = x0.x, a.w[4 * j + 1] = x0.y, a.w[4 * j + 2] = x0.z, a.w[4 * j + 3] = x0.w;
                    b.w[4 * j] = x1.x, b.w[4 * j + 1] = x1.y, b.w[4 * j + 2] = x1.z, b.w[4 * j + 3] = x1.w;
                }
                encode_unit(a, b, block_mag(a), block_mag(b), row_scales[rr], given, q, s, r0 + rr < R);
            }
        }
        // lane: group of 32 rows (lane % 8) and column pair (lane / 8 of the warp's four)
        const int group = threadIdx.x & 7, pair = threadIdx.x >> 3;
        const int64_t c = c0 + 2 * pair;
        const unsigned char* column = piece_at(32 * group, 2 * pair / kPer) + (2 * pair % kPer) * (int)sizeof(T);
        uint2 codes[2][2];
        uint32_t sb[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[2][16];
            uint32_t m[2] = {0u, 0u};
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 f = *reinterpret_cast<const float2*>(column + (16 * h + j) * kPitch);
                    v[0][j] = f.x, v[1][j] = f.y;
                    m[0] = mag_max<T>(m[0], __float_as_uint(f.x));
                    m[1] = mag_max<T>(m[1], __float_as_uint(f.y));
                }
            } else {
                uint32_t both = 0u;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(column + (16 * h + j) * kPitch);
                    both = mag_max<T>(both, w);
                    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                        v[0][j] = __uint_as_float(w << 16), v[1][j] = __uint_as_float(w & 0xffff0000u);
                    } else {
                        const float2 f = h2_to_f2(w);
                        v[0][j] = f.x, v[1][j] = f.y;
                    }
                }
                m[0] = mag_f32<T>(both & 0xffffu), m[1] = mag_f32<T>(both & 0xffff0000u);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const RowScale rs = col_scales[2 * pair + e];
                sb[e][h] = !given && rs.y != 0.f ? encode_block<T, true>(v[e], __uint_as_float(m[e]), rs, false, codes[e][h])
                                                 : encode_block<T, false>(v[e], __uint_as_float(m[e]), rs, given, codes[e][h]);
            }
        }
        // the tile's 64 columns lie in one 128-row block of the column operand, its 256 rows in one code tile
        uint8_t* q = cols.q + ((c0 >> 7) * (Rp >> 8) + (r0 >> 8)) * 16384;
        uint8_t* s = cols.s + ((c0 >> 7) * (Rp >> 6) + (r0 >> 6)) * 512;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t word = sb[e][0] | (sb[e][1] << 8);
            word |= __shfl_down_sync(0xffffffffu, word, 1) << 16;  // two groups: the four scales of a word
            if (c + e >= C) continue;
            const uint32_t in = ((uint32_t)c0 & 64u) + 2 * pair + e;
            *reinterpret_cast<uint4*>(q + unit_codes(in, group)) = make_uint4(codes[e][0].x, codes[e][0].y, codes[e][1].x, codes[e][1].y);
            if ((group & 1) == 0) *reinterpret_cast<uint32_t*>(s + unit_scales(in, group)) = word;
        }
        __syncthreads();  // the buffer and the scales are free
    }
}

template <typename T>
cudaError_t quantize(const T* x, int64_t R, int64_t C, int64_t ld, const moe_nvfp4_operand* rows,
                     const moe_nvfp4_operand* cols, bool given, unsigned* maxima, cudaStream_t st) {
    bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
    if (!cols) {
        const int64_t units = pad_to(C, 256) / 32;
        int tpr_log = 5;  // the fewest threads that hold a row, 32 elements each
        while ((1 << tpr_log) < kThreads && (1 << tpr_log) < units) ++tpr_log;
        const int64_t per = kThreads >> tpr_log, grid = (R + per - 1) / per;
        bool gr = rows->gs_rows != 0;
        uint8_t *q = rows->q, *s = rows->s;
        float* gs = rows->gs;
        constexpr int kCtas = sizeof(T) == 4 ? 3 : 4;
        const int64_t resident = sm_count() * kCtas;
        // (us, streamed / not: aligned rows 4096 x 8192 18.4 / 19.3, 16384 x 512 9.2 / 9.6, but two waves or less, 8192 x 1024, 6.0 / 4.6;
        // others 4096 x 8191 24.6 / 64, 8192 x 700 10.1 / 12.8, but half a warp's units, 8192 x 257, 10.2 / 6.8)
        if (units <= kThreads && (wide ? grid > 2 * resident : units > 16)) {
            const void* f = wide ? (const void*)nvfp4_rows_stream_kernel<T, kCtas, true> : (const void*)nvfp4_rows_stream_kernel<T, kCtas, false>;
            const size_t smem = 2 * (kThreads / 32) * (size_t)(wide ? stream_warp_bytes<T, true>() : stream_warp_bytes<T, false>());
            void* args[] = {&x, &R, &C, &ld, &tpr_log, &q, &s, &gs, &given, &gr};
            return launch_kernel(f, dim3((unsigned)(grid < resident ? grid : resident)), dim3(kThreads), smem, st, true, args);
        }
        void* args[] = {&x, &R, &C, &ld, &wide, &tpr_log, &q, &s, &gs, &given, &gr};
        return launch_kernel((const void*)nvfp4_rows_kernel<T>, dim3((unsigned)grid), dim3(kThreads), 0, st, true, args);
    }
    unsigned* row_max = rows ? maxima : nullptr;
    unsigned* col_max = maxima + (rows ? R : 0);
    if (!given) {
        int64_t n = (rows ? R : 0) + C;
        void* zero_args[] = {&maxima, &n};
        cudaError_t e = launch_kernel((const void*)nvfp4_zero_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                                      true, zero_args);
        if (e != cudaSuccess) return e;
        const int warp_cols = 32 * 16 / (int)sizeof(T);
        int ct = (int)((C + warp_cols - 1) / warp_cols);
        const int64_t grid = ct * ((R + kThreads / 32 * kMaxRows - 1) / (kThreads / 32 * kMaxRows));
        void* args[] = {&x, &R, &C, &ld, &wide, &ct, &row_max, &col_max};
        e = launch_kernel((const void*)nvfp4_maxima_kernel<T>, dim3((unsigned)grid), dim3(kThreads), 0, st, true, args);
        if (e != cudaSuccess) return e;
    }
    // the padded contractions: columns to 256 for the row form, rows to 256 for the column form
    int ct = (int)(pad_to(C, rows ? 256 : kTileC) / kTileC);
    const int64_t rt = pad_to(R, 256) / kTileR;
    moe_nvfp4_operand a = rows ? *rows : moe_nvfp4_operand{nullptr, nullptr, nullptr, 0}, b = *cols;
    int n_tiles = (int)(ct * rt);
    const int resident = sm_count() * (sizeof(T) == 4 ? 1 : 3);
    void* args[] = {&x, &R, &C, &ld, &wide, &ct, &n_tiles, &row_max, &col_max, &a, &b, &given};
    return launch_kernel((const void*)nvfp4_both_kernel<T>, dim3((unsigned)(n_tiles < resident ? n_tiles : resident)), dim3(kThreads),
                         (size_t)2 * kTileR * kTileC * sizeof(T), st, true, args);
}

// Values of an operand: (E2M1 * E4M3) * row scale, the exact product of the first two rounded once.
__global__ void __launch_bounds__(kThreads)
    nvfp4_values_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, const float* __restrict__ gs, bool gs_rows,
                        int64_t R, int64_t K, float* __restrict__ v) {
    const int64_t units = (K + 31) / 32, Kp = pad_to(K, 256);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < R * units; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / units, u = i % units;
        const uint4 c = *reinterpret_cast<const uint4*>(q + mma_tile_offset(r, u, Kp));
        const float2 sc = e4m3x2_to_f2(*reinterpret_cast<const uint16_t*>(s + mma_scale_offset(r, 2 * u, 2 * Kp)));
        const float g = gs[gs_rows ? r : 0];
        const uint32_t words[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            uint32_t h[4];
            e2m1x8_to_h2(words[m], h);
            const float sv = m < 2 ? sc.x : sc.y;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 p = h2_to_f2(h[j / 2]);
                const int64_t k = 32 * u + 8 * m + j;
                if (k < K) v[r * K + k] = __fmul_rn(__fmul_rn(j & 1 ? p.y : p.x, sv), g);
            }
        }
    }
}

}  // namespace

cudaError_t launch_nvfp4_quantize(const void* x, moe_dtype dtype, int64_t R, int64_t C, int64_t ld,
                                  const moe_nvfp4_operand* rows, const moe_nvfp4_operand* cols, bool given, void* maxima,
                                  cudaStream_t st) {
    if (R == 0 || C == 0) return cudaSuccess;
    unsigned* m = static_cast<unsigned*>(maxima);
    if (dtype == MOE_F32) return quantize(static_cast<const float*>(x), R, C, ld, rows, cols, given, m, st);
    if (dtype == MOE_BF16) return quantize(static_cast<const __nv_bfloat16*>(x), R, C, ld, rows, cols, given, m, st);
    return quantize(static_cast<const __half*>(x), R, C, ld, rows, cols, given, m, st);
}

cudaError_t launch_nvfp4_values(const moe_nvfp4_operand* op, int64_t R, int64_t K, float* v, cudaStream_t st) {
    if (R == 0 || K == 0) return cudaSuccess;
    const int64_t n = R * ((K + 31) / 32);
    int64_t blocks = (n + kThreads - 1) / kThreads;
    if (blocks > 152 * 64) blocks = 152 * 64;
    nvfp4_values_kernel<<<(unsigned)blocks, kThreads, 0, st>>>(op->q, op->s, op->gs, op->gs_rows != 0, R, K, v);
    return cudaGetLastError();
}

}  // namespace moe
