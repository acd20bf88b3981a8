// Rows of tokens with the channels last: neighbouring channels of a row in registers, and the
// pieces that sequences are cut into.
#pragma once

#include "kda_layer.h"
#include "kda_ops.cuh"

namespace kda {
namespace rows {

// The debug build's check of an index (dbg_ok()).  Where its caller has set KDA_DBG_SHORT in the flag word, every
// extent counts as one less, so that the checks of the last elements report.
constexpr unsigned DBG_SHORT = 8u;
__device__ __forceinline__ bool in_bounds(unsigned *flags, size_t idx, size_t n, unsigned bit) {
#ifdef KDA_DEBUG_CHECKS
    return dbg_ok(flags, idx + (flags && *(volatile unsigned *)flags & DBG_SHORT ? 1 : 0), n, bit);
#else
    return true;
#endif
}

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half from_f32<__half>(float x) {
    return __float2half_rn(x);
}

// Neighbouring elements as FP32 and back, two at a time.
__device__ __forceinline__ float2 get_two(const float *p) { return make_float2(p[0], p[1]); }
__device__ __forceinline__ float2 get_two(const __nv_bfloat16 *p) {
    const uint32_t u = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 get_two(const __half *p) {
    return __half22float2(*reinterpret_cast<const __half2 *>(p));
}
__device__ __forceinline__ void set_two(float *p, float2 x) {
    p[0] = x.x;
    p[1] = x.y;
}
__device__ __forceinline__ void set_two(__nv_bfloat16 *p, float2 x) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(x);
}
__device__ __forceinline__ void set_two(__half *p, float2 x) {
    *reinterpret_cast<__half2 *>(p) = __float22half2_rn(x);
}

// V neighbouring channels of a row.
template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
    T v[V];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = from_f32<T>(0.f);
    }
    __device__ __forceinline__ float operator[](int i) const { return as_f32(v[i]); }
    // (even i)
    __device__ __forceinline__ float2 two(int i) const { return get_two(v + i); }
    __device__ __forceinline__ void put(int i, float2 x) { set_two(v + i, x); }
};

// An element of a parameter, whose type may be x's or FP32.
__device__ __forceinline__ float param(const void *p, int dtype, size_t i, float none) {
    if (!p) return none;
    if (dtype == TYPE_FP32) return ((const float *)p)[i];
    if (dtype == TYPE_BF16) return as_f32(((const __nv_bfloat16 *)p)[i]);
    return as_f32(((const __half *)p)[i]);
}

// 1 / (1 + e^-x), from the exponential and reciprocal units (2^-22 each); 0 and 1 at the far ends.
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }
// d silu / dx, with s = sigmoid(x)
__device__ __forceinline__ float silu_slope(float x, float s) { return s * fmaf(x, 1.f - s, 1.f); }

// A piece of a sequence: its tokens [begin, begin + len) of the sequence's [0, total).
struct Piece {
    long long row0;  // the sequence's first row
    int seq, index, begin, len, total;
};

// Piece p of the pieces of `size` tokens.  Packed sequences take theirs from cu[n] / size + n on, so
// that no two meet and T / size + num_seqs cover every input; each has one at least, an empty
// sequence too.  len < 0: there is none.
__device__ __forceinline__ Piece find_piece(const Tokens &t, long long p, int size) {
    Piece x;
    if (!t.cu_seqlens) {
        const int per = t.T > size ? (t.T + size - 1) / size : 1;
        x.seq = (int)(p / per);
        x.index = (int)(p - (long long)x.seq * per);
        x.row0 = (long long)x.seq * t.T;
        x.total = t.T;
    } else {
        auto token = [&](int v) { return v < 0 ? 0 : v > t.T ? t.T : v; };
        // the last sequence whose pieces begin at or before this one, by 32 of them at a time: a step
        // waits for memory once
        int lo = 0, n = t.num_seqs;
        const int lane = threadIdx.x & 31;
        while (n > 1) {
            const int step = (n + 31) / 32, at = lo + lane * step;
            const bool before = lane * step < n && (lane == 0 || token(t.cu_seqlens[at]) / size + at <= p);
            const unsigned mask = __ballot_sync(0xffffffffu, before);
            const int last = mask == 0xffffffffu ? 31 : __ffs(~mask) - 2;
            lo += last * step;
            n = min(step, n - last * step);
        }
        const int a = token(t.cu_seqlens[lo]), b = token(t.cu_seqlens[lo + 1]);
        x.seq = lo;
        x.row0 = a;
        x.total = b > a ? b - a : 0;
        x.index = (int)(p - (a / size + lo));
    }
    x.begin = x.index * size;
    const int left = x.total - x.begin;
    x.len = x.index < 0 || (left <= 0 && x.index > 0) ? -1 : left < size ? left : size;
    return x;
}

inline bool aligned(const void *p, size_t to) { return (uintptr_t)p % to == 0; }

// The widest of 16, 8, 4 bytes and an element on whose boundaries all rows and blocks of `per` channels
// begin.
struct Boundary {
    int es, unit;
    Boundary(int es, int per) : es(es), unit(16) {
        while (unit > es && (long long)per * es % unit) unit /= 2;
    }
    void add(const void *p, long long stride) {
        while (p && unit > es && !(aligned(p, unit) && stride * es % unit == 0)) unit /= 2;
    }
};

// Eight neighbouring channels of a token on their way into shared memory, `unit` bytes at a time (16,
// 8 or 4 by asynchronous copies, or an element): rows and blocks of channels begin on such
// boundaries.  Zeros where there are none (from `left` on, or without ok).
template <typename T>
__device__ __forceinline__ void fetch_chunk(Vec<T, 8> *slot, const void *base, const T *from, int left,
                                            bool ok, int unit) {
    const char *at = (const char *)from;  // (not looked at unless ok; base is any address that may be)
    constexpr int E = sizeof(T);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot);
    if (unit == 16) {
#pragma unroll
        for (int i = 0; i < 8 * E; i += 16) {
            const bool in = ok && i < left * E;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i), "l"(in ? at + i : base),
                         "r"(in ? 16 : 0) : "memory");
        }
    } else if (unit == 8) {
#pragma unroll
        for (int i = 0; i < 8 * E; i += 8) {
            const bool in = ok && i < left * E;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + i), "l"(in ? at + i : base),
                         "r"(in ? 8 : 0) : "memory");
        }
    } else if (unit == 4) {
#pragma unroll
        for (int i = 0; i < 8 * E; i += 4) {
            const bool in = ok && i < left * E;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + i), "l"(in ? at + i : base),
                         "r"(in ? 4 : 0) : "memory");
        }
    } else {
        T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = ok && i < left ? ((const T *)at)[i] : from_f32<T>(0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) slot->v[i] = v[i];
    }
}

}  // namespace rows
}  // namespace kda
