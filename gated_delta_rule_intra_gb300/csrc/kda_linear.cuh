// Shared parts of the matrix product's kernels.
#pragma once

#include "kda_rows.cuh"

namespace kda {
namespace linear {

using namespace rows;

// Polls of a bounded wait, behind which the kernel gives up (and writes NaN).  In the debug build it may be told
// to give up at once (kda_debug_set_give_up): none or all, because a pair's CTAs have asked for the same
// copies then, as many as there are stages, and the first one's last waits, which are never shortened, see
// them land.
constexpr uint32_t kWaitPolls = 1u << 22;
__device__ __forceinline__ uint32_t wait_polls(bool give_up) {
#ifdef KDA_DEBUG_CHECKS
    return give_up ? 0 : kWaitPolls;
#else
    return kWaitPolls;
#endif
}

// erfc(|x| / sqrt 2) of two values.  With z = |x| / sqrt 2 and t = 1 / (1 + z / 2), log2(erfc(z) e^(z^2) / t)
// is a smooth function of t on [0, 1]: its Chebyshev interpolation of degree 7 (nodes on z <= 9.5, behind
// which e^(-z^2) is nothing), in powers of t.  Relative error 7e-7 before the exponential's own rounding
// (7e-6 at |x| = 9): Phi keeps its accuracy in the negative tail, which 1 + erf(x) would lose, at a
// third of the library function's instructions.
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 erfc_abs(float2 x) {
    const float2 a = make_float2(fabsf(x.x), fabsf(x.y)), w = fma2(a, twice(0.35355339f), twice(1.f));
    const float2 t = make_float2(rcp(w.x), rcp(w.y));
    float2 r = fma2(t, twice(-0.270080537f), twice(1.08023681f));
    r = fma2(t, r, twice(-1.43607122f));
    r = fma2(t, r, twice(0.496005889f));
    r = fma2(t, r, twice(-0.0518293115f));
    r = fma2(t, r, twice(0.566456863f));
    r = fma2(t, r, twice(1.44100291f));
    r = fma2(t, r, twice(-1.82572244f));
    r = fma2(mul2(a, twice(-0.72134752f)), a, r);  // -z^2 log2(e)
    return mul2(t, make_float2(ex2(r.x), ex2(r.y)));
}
// Beyond +-64 Phi is 0 or 1 and its product with x is taken as that of 64 (0 times infinity).
__device__ __forceinline__ float near(float x) { return fminf(fmaxf(x, -64.f), 64.f); }
__device__ __forceinline__ float2 gelu(float2 x) {
    const float2 q = erfc_abs(x);  // x Phi(x) = max(x, 0) - |x| q / 2
    return make_float2(fmaf(-0.5f * fabsf(near(x.x)), q.x, fmaxf(x.x, 0.f)),
                       fmaf(-0.5f * fabsf(near(x.y)), q.y, fmaxf(x.y, 0.f)));
}
__device__ __forceinline__ float2 gelu_slope(float2 x) {  // Phi(x) + x phi(x)
    const float2 q = mul2(erfc_abs(x), twice(0.5f)), y = make_float2(near(x.x), near(x.y));
    const float2 e = mul2(mul2(y, twice(-0.72134752f)), y);
    const float2 phi = make_float2(x.x < 0.f ? q.x : 1.f - q.x, x.y < 0.f ? q.y : 1.f - q.y);
    return fma2(mul2(y, twice(0.39894228f)), make_float2(ex2(e.x), ex2(e.y)), phi);
}
__device__ __forceinline__ float finite(float x) { return fminf(fmaxf(x, -3.4028235e38f), 3.4028235e38f); }
__device__ __forceinline__ float2 sigmoid2(float2 x) { return make_float2(sigmoid(x.x), sigmoid(x.y)); }

template <int ACT> __device__ __forceinline__ float2 activate(float2 x) {
    if constexpr (ACT == ACT_SILU) return mul2(x, sigmoid2(x));
    if constexpr (ACT == ACT_GELU) return gelu(x);
    if constexpr (ACT == ACT_RELU) return make_float2(x.x < 0.f ? 0.f : x.x, x.y < 0.f ? 0.f : x.y);
    return x;
}
__device__ __forceinline__ float activate(float x, int act) {
    const float2 p = twice(x);
    return act == ACT_SILU ? activate<ACT_SILU>(p).x : act == ACT_GELU ? activate<ACT_GELU>(p).x
           : act == ACT_RELU ? activate<ACT_RELU>(p).x : x;
}
// d act / dx; 0 in relu's corner.
__device__ __forceinline__ float2 slope(float2 x, int act) {
    if (act == ACT_SILU) {
        // (x may be infinite where the sum was beyond the 16-bit type: with the largest finite number beside 1 - s
        // the ends are 0 and 1 instead of 0 times infinity; NaN stays, by s)
        const float2 s = sigmoid2(x), y = make_float2(finite(x.x), finite(x.y));
        return mul2(s, fma2(y, fma2(s, twice(-1.f), twice(1.f)), twice(1.f)));
    }
    if (act == ACT_GELU) return gelu_slope(x);
    auto step = [](float v) { return v > 0.f ? 1.f : v == v ? 0.f : v; };
    return act == ACT_RELU ? make_float2(step(x.x), step(x.y)) : twice(1.f);
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
