// Shared parts of the layer-norm kernels: a row is held in registers by a group of TPR threads
// (the smallest power of two that holds it).  A thread has 32 bytes of it: with 16, BF16 rows are
// bound by instructions, most of them in the sums over lanes (32768 x 2048: forward 54.5 us with
// 76% of the issue slots taken).  Rows on no 16-byte boundary take eight elements a thread, which
// need more registers each.
#pragma once

#include "kda_ops.cuh"

namespace kda {
namespace norm {

constexpr int kMaxWidth = 8192;  // widest row that one CTA holds in registers
template <typename T, bool WIDE> constexpr int elements() {  // of a thread
    return WIDE ? 32 / (int)sizeof(T) : 8;
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

// Neighbouring elements as FP32.
__device__ __forceinline__ float2 two(const float *p) { return make_float2(p[0], p[1]); }
__device__ __forceinline__ float2 two(const __nv_bfloat16 *p) {
    const uint32_t u = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 two(const __half *p) {
    return __half22float2(*reinterpret_cast<const __half2 *>(p));
}
__device__ __forceinline__ void put_two(float *p, float2 x) {
    p[0] = x.x;
    p[1] = x.y;
}
__device__ __forceinline__ void put_two(__nv_bfloat16 *p, float2 x) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(x);
}
__device__ __forceinline__ void put_two(__half *p, float2 x) {
    *reinterpret_cast<__half2 *>(p) = __float22half2_rn(x);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Where a row is in its tensor of `end` elements, from the first to behind the last, for the debug
// build's checks.
struct Place {
    unsigned *dbg;
    size_t at, end;
    __device__ __forceinline__ Place(const NormArgs &a, long long row, long long stride)
        : dbg(a.dbg), at((size_t)row * stride), end((size_t)(a.rows - 1) * stride + a.width) {}
    __device__ __forceinline__ bool ok(int last, unsigned bit) const {
        return dbg_ok(dbg, at + last, end, bit);
    }
};

// A thread's elements of a row.  WIDE: 16-byte accesses, a group's next to each other; otherwise
// single elements TPR columns apart (rows that start at no 16-byte boundary).
template <typename T, bool WIDE, int TPR> struct Part {
    static constexpr int E = elements<T, WIDE>(), kVec = 16 / (int)sizeof(T);
    alignas(16) T v[E];

    static __device__ __forceinline__ int col(int t, int i) {
        return WIDE ? (i / kVec * TPR + t) * kVec + i % kVec : t + i * TPR;
    }

    // (rows on 16-byte boundaries come through Stream)
    __device__ __forceinline__ void load(const T *row, int t, int width, bool ok,
                                         const Place &where) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            v[i] = ok && col(t, i) < width && where.ok(col(t, i), DBG_LOAD) ? row[col(t, i)]
                                                                           : from_f32<T>(0.f);
    }
    __device__ __forceinline__ void store(T *row, int t, int width, bool ok,
                                          const Place &where) const {
        if (WIDE) {
#pragma unroll
            for (int i = 0; i < E; i += kVec)
                if (ok && col(t, i) < width && where.ok(col(t, i) + kVec - 1, DBG_STORE))
                    *reinterpret_cast<uint4 *>(row + col(t, i)) =
                        *reinterpret_cast<const uint4 *>(&v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (ok && col(t, i) < width && where.ok(col(t, i), DBG_STORE))
                    row[col(t, i)] = v[i];
        }
    }
};

// Rows on their way to a thread: its two 16-byte parts of each of the next DEPTH - 1 rows, copied
// asynchronously into slots of its own in shared memory, so that as many bytes are in flight as
// the memory's latency asks for without a register or a barrier.  Rows on no
// 16-byte boundary (WIDE false) come through registers, one row ahead.
template <typename T, bool WIDE, int TPR, int THREADS, int DEPTH> struct Stream {
    using P = Part<T, WIDE, TPR>;
    static constexpr int kParts = 2;
    static constexpr int kBytes = WIDE ? DEPTH * kParts * THREADS * 16 : 0;
    uint4 *slots;  // [DEPTH][kParts][THREADS], this thread's column
    P next;

    __device__ __forceinline__ Stream(char *s)
        : slots(reinterpret_cast<uint4 *>(s) + threadIdx.x) {}
    __device__ __forceinline__ void fetch(int stage, const T *row, int t, int width, bool ok,
                                          const Place &where) {
        if (WIDE) {
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const int c = P::col(t, i * P::kVec);
                const bool in = ok && c < width && where.ok(c + P::kVec - 1, DBG_LOAD);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(
                                     slots + (stage * kParts + i) * THREADS)),
                             "l"(in ? row + c : row), "r"(in ? 16 : 0)
                             : "memory");
            }
        } else {
            next.load(row, t, width, ok, where);
        }
    }
    __device__ __forceinline__ P take(int stage) {
        if constexpr (!WIDE) {
            return next;
        } else {
            P p;
#pragma unroll
            for (int i = 0; i < kParts; ++i)
                *reinterpret_cast<uint4 *>(&p.v[i * P::kVec]) =
                    slots[(stage * kParts + i) * THREADS];
            return p;
        }
    }
};

// An element of weight or bias, whose type may be x's or FP32.
__device__ __forceinline__ float param(const void *p, int dtype, int c, float none) {
    if (!p) return none;
    if (dtype == NORM_FP32) return ((const float *)p)[c];
    if (dtype == NORM_BF16) return as_f32(((const __nv_bfloat16 *)p)[c]);
    return as_f32(((const __half *)p)[c]);
}

// Rows that a group takes at once in the forward: two where their sums cross warps, each covering
// the other's exchange (32768 x 2048 BF16 45 us, one at a time 59; inside a warp there is no
// difference: 524288 x 128 takes 45 us either way).
template <bool WIDE, int TPR> constexpr int at_once() { return WIDE && TPR >= 64 ? 2 : 1; }

template <int TPR> constexpr int threads() { return TPR < 256 ? 256 : TPR; }

// Barrier of one row's group of threads (TPR > 32).
template <int TPR> __device__ __forceinline__ void group_sync(int group) {
    if (threads<TPR>() == TPR)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
}

template <int N> __device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int off = N / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

inline int esize(int dtype) { return dtype == NORM_FP32 ? 4 : 2; }

// Threads of a row, e elements each; 0 when one CTA's registers do not hold it.
inline int group_of(int width, int e) {
    if (width > kMaxWidth) return 0;
    int t = 128 / e;
    while (t * e < width) t *= 2;
    return t;
}

inline bool wide_ok(int dtype, int width, const void *p, long long stride, bool with = true) {
    const int vec = 16 / esize(dtype);
    return !with || (width % vec == 0 && (uintptr_t)p % 16 == 0 && stride % vec == 0);
}

}  // namespace norm
}  // namespace kda
