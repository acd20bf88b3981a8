// Checks of arguments that the C entry points share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#pragma GCC visibility push(default)
#include "kda.h"
#pragma GCC visibility pop

namespace kda {
kda_status_t require_device();  // kda_api.cu
unsigned *debug_flags();
bool debug_give_up();

// Bytes that a call reads or writes: one run, or rows of `row` bytes `step` apart.
struct Range {
    uintptr_t lo, hi, row, step;
    Range(const void *p, size_t bytes)
        : lo((uintptr_t)p), hi(p ? (uintptr_t)p + bytes : 0), row(bytes), step(bytes) {}
    Range(const void *p, long long rows, int width, long long stride, int es)
        : Range(p, rows ? ((size_t)(rows - 1) * stride + width) * es : 0) {
        row = (size_t)width * es;
        step = (size_t)stride * es;
    }
};

inline bool meet(const Range &a, const Range &b) {
    if (!(a.lo < b.hi && b.lo < a.hi)) return false;
    if (a.step != b.step) return true;
    // rows equally far apart may lie between each other's (column slices of one buffer)
    const uintptr_t off = b.lo >= a.lo ? (b.lo - a.lo) % a.step
                                       : (a.step - (a.lo - b.lo) % a.step) % a.step;
    return !(off >= a.row && off + b.row <= a.step);
}

// Every output against every input and every other output.
template <size_t NO, size_t NI> inline bool overlap(const Range (&out)[NO], const Range (&in)[NI]) {
    for (size_t o = 0; o < NO; ++o) {
        for (const Range &r : in)
            if (meet(out[o], r)) return true;
        for (size_t p = o + 1; p < NO; ++p)
            if (meet(out[o], out[p])) return true;
    }
    return false;
}

template <size_t N> bool misaligned(const void *const (&ps)[N], unsigned to) {
    for (const void *p : ps)
        if ((uintptr_t)p % to) return true;
    return false;
}

inline kda_status_t finish(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace kda
