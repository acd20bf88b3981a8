// Device helpers of the recurrence and layer-norm kernels, next to those of kda_common.cuh.
#pragma once

#include "kda_common.cuh"
#include "kda_ops.h"

namespace kda {

// Kernels launched with launch_early() may start before the one in front of them on the stream has
// ended, so that the launch itself overlaps its tail (a prefill of 37 tokens 10.2 -> 7.3 us, the
// three launches of a 2021 x 1111 layer norm 22.9 -> 16.9).  Each thread's first act there is
// wait_for_previous(): everything in front is complete and its writes are visible behind it.  No
// CTA may leave this out, one with nothing to do included: the next kernel's wait covers what is
// in front of this one only through this one.  The backward's long kernels are launched as usual:
// early, their CTAs land on other SMs than the ones that wrote what they read (1655 -> 1678 us
// for a training step).
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t stream, Args... args) {
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Two FP32 operations in one instruction (the pair in a 64-bit register).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
        "mul.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
        "add.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
        "mov.b64 z, {%6, %7};\nfma.rn.f32x2 z, x, y, z;\nmov.b64 {%0, %1}, z;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// All but the N newest groups of this thread's copies have landed.
template <int N> __device__ __forceinline__ void cp_async_wait_newest() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace kda
