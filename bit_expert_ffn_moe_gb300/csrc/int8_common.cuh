// int8_common.cuh -- what the kernels of the 8-bit products share.
#pragma once

#include "ops.cuh"

namespace moe {

template <typename T>
__device__ __forceinline__ T int8_result(float v);
template <>
__device__ __forceinline__ float int8_result<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 int8_result<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half int8_result<__half>(float v) { return __float2half_rn(v); }

// silu(gate) up.  For a negative gate exp(gate) as a square, one factor on either side, so that neither it nor exp(-gate) leaves fp32's
// range before the result does.
__device__ __forceinline__ float int8_gated(float gate, float up) {
    const float e = expf(gate < 0.f ? 0.5f * gate : -gate);
    return gate < 0.f ? (gate * e) * (up * e) / (1.f + e * e) : gate / (1.f + e) * up;
}

// ------------------------------------------------------------------ rows in 8 bits
// The bits of |v|: NaN above infinity above all numbers.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct Scale {
    float s, inverse;
    bool bad, sure;  // with a NaN or an infinity; neither the scale nor remainders lose bits to the range
};
__device__ __forceinline__ Scale scale_of(uint32_t most) {
    Scale r;
    r.bad = most >= 0x7f800000u;
    r.s = __fdiv_rn(__uint_as_float(most), 127.f);
    if (!(r.s > 0.f)) r.s = 1.f;
    r.inverse = 1.f / r.s;
    r.sure = !r.bad && r.s > 0x1p-80f && r.s < 0x1p100f;
    if (r.bad) r.s = __uint_as_float(0x7fffffffu);
    return r;
}
// v / s, rounded to fp32, rounded to a whole number, by the division.
static __device__ __noinline__ float whole(float v, float s, bool bad) {
    return bad ? 0.f : fminf(fmaxf(rintf(__fdiv_rn(v, s)), -127.f), 127.f);
}
// The same of eight values.  The product with the reciprocal (correctly rounded) is within two steps of the quotient; correcting it by its
// remainder, which an fma gives, makes it one of the quotient's two neighbours, and correcting that once more the quotient rounded to
// fp32 (Markstein 1990).  Quotients of 16-bit numbers are halves of whole numbers often enough that a test for these, with the division
// behind it, took twice as long.  Adding 1.5 x 2^23 rounds to a whole number, ties to even.
__device__ __forceinline__ void whole8(const float (&v)[8], const Scale& s, float (&q)[8]) {
    if (s.sure) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float t = v[i] * s.inverse;
            t = fmaf(fmaf(-t, s.s, v[i]), s.inverse, t);
            t = fmaf(fmaf(-t, s.s, v[i]), s.inverse, t);
            q[i] = (t + 12582912.f) - 12582912.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = whole(v[i], s.s, s.bad);
    }
}

template <typename T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value<float>(float v) { return v; }
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float value<__half>(__half v) { return __half2float(v); }

// The larger of the magnitudes in m and the magnitude of w, of 16-bit numbers in both halves; NaN above all.
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t w);
template <>
__device__ __forceinline__ uint32_t larger<float>(uint32_t m, uint32_t w) { return max(m, w & 0x7fffffffu); }
template <>
__device__ __forceinline__ uint32_t larger<__nv_bfloat16>(uint32_t m, uint32_t w) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t larger<__half>(uint32_t m, uint32_t w) {
    const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&m), __habs2(*reinterpret_cast<const __half2*>(&w)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ float2 two(uint32_t w);
template <>
__device__ __forceinline__ float2 two<__nv_bfloat16>(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
template <>
__device__ __forceinline__ float2 two<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Values c .. c + 7 of a row of K as they come, zeros behind its end.  WIDE: rows that start on 16 bytes.
template <typename T>
struct Eight {
    static constexpr int kWords = 2 * (int)sizeof(T);
    uint32_t w[kWords];

    template <bool WIDE>
    __device__ __forceinline__ void load(const T* row, int64_t c, int64_t K) {
        if (WIDE && c + 8 <= K) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + c) + i);
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = c + i < K ? __ldg(reinterpret_cast<const uint32_t*>(row + c + i)) : 0;
        } else {
            // whole words, shifted where the row begins in the middle of one; of those that begin behind the row's end the last one again
            const uintptr_t at = reinterpret_cast<uintptr_t>(row + min(c, K - 1)), end = reinterpret_cast<uintptr_t>(row + K - 1) & ~(uintptr_t)3;
            const uint32_t shift = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 2) * 8;
            uint32_t u[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) u[i] = __ldg(reinterpret_cast<const uint32_t*>(min((at & ~(uintptr_t)3) + 4 * i, end)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = __funnelshift_r(u[i], u[i + 1], shift);
                const int64_t left = K - c - 2 * i;
                w[i] = left >= 2 ? w[i] : left == 1 ? w[i] & 0xffffu : 0;
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    // The larger of `most` and its magnitudes; 16-bit ones in halves.
    __device__ __forceinline__ uint32_t most(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) m = larger<T>(m, w[i]);
        return m;
    }
    // That of a row, as the bits of an fp32 number (NaN above infinity above all numbers).
    __device__ __forceinline__ static uint32_t as_fp32(uint32_t m) {
        if constexpr (sizeof(T) == 4) return m;
        else {
            const float2 v = two<T>(m);
            return max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                const float2 v = two<T>(w[i]);
                f[2 * i] = v.x, f[2 * i + 1] = v.y;
            }
        }
    }
};

// Where expert e's rows start; offsets of other rows than these lead nowhere outside them.
__device__ __forceinline__ int64_t int8_offset(const Int8ProductArgs& a, int e) {
    return min(max((int64_t)__ldcg(a.offsets + e), (int64_t)0), a.M);
}

// Few rows: of the operand, or, where x is not null, [..][ldx] of x_dtype, quantised by every CTA for itself (K at most kInt8DotK); with
// inv [T][k], M = T k at most 32, row inv[t k + j] is row t of x.
constexpr int kInt8DotK = 16384;
cudaError_t launch_int8_dot(const Int8ProductArgs& a, moe_dtype dtype, bool gated, const void* x, moe_dtype x_dtype, int64_t ldx,
                            const int32_t* inv, int k, cudaStream_t st);
// A few dozen rows with one matrix, where its tiles do not outnumber the SMs.
bool int8_few_fits(const Int8ProductArgs& a);
cudaError_t launch_int8_few(const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st);
cudaError_t launch_int8_mma(const Int8ProductArgs& a, moe_dtype dtype, bool gated, bool pair, cudaStream_t st);

}  // namespace moe
