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

cudaError_t launch_int8_dot(const Int8ProductArgs& a, moe_dtype dtype, bool gated, cudaStream_t st);
cudaError_t launch_int8_mma(const Int8ProductArgs& a, moe_dtype dtype, bool gated, bool pair, cudaStream_t st);

}  // namespace moe
