// Shared parts of the matrix product's kernels.
#pragma once

#include "kda_rows.cuh"

namespace kda {
namespace linear {

using namespace rows;

__device__ __forceinline__ float activate(float x, int act) {
    if (act == ACT_SILU) return x * sigmoid(x);
    if (act == ACT_GELU) return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
    if (act == ACT_RELU) return x < 0.f ? 0.f : x;
    return x;
}
// d act / dx; of relu's corner 0.
__device__ __forceinline__ float slope(float x, int act) {
    if (act == ACT_SILU) return silu_slope(x, sigmoid(x));
    if (act == ACT_GELU)
        return fmaf(x * 0.39894228040143268f, ex2(-0.72134752044448170f * x * x),
                    0.5f * (1.f + erff(x * 0.70710678118654752f)));
    if (act == ACT_RELU) return x > 0.f ? 1.f : x == x ? 0.f : x;
    return 1.f;
}

// Two values as a pair of 16-bit ones.
template <typename T> __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    if (sizeof(T) && std::is_same<T, __half>::value)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <typename T> __device__ __forceinline__ float2 unpack(uint32_t x) {
    if (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

}  // namespace linear
}  // namespace kda
