// Shared parts of the short causal convolution's kernels.
//   pre[t, d] = bias[d] + sum_j weight[d, j] x[t - W + 1 + j, d],  y = act(pre),
// over the tokens of a sequence; what lies in front of it comes from its state, the W - 1 inputs
// before its first token, oldest first (zeros without one).
#pragma once

#include "kda_rows.cuh"

namespace kda {
namespace conv {

using namespace rows;

// acc += x * y, two channels in one instruction.
template <int V> __device__ __forceinline__ void vfma(float (&acc)[V], const float (&x)[V], const float (&y)[V]) {
    if constexpr (V == 1) {
        acc[0] = fmaf(x[0], y[0], acc[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 r = fma2(make_float2(x[i], x[i + 1]), make_float2(y[i], y[i + 1]),
                                  make_float2(acc[i], acc[i + 1]));
            acc[i] = r.x;
            acc[i + 1] = r.y;
        }
    }
}
template <typename T, int V> __device__ __forceinline__ void widen(float (&f)[V], const Vec<T, V> &x) {
    if constexpr (V == 1) {
        f[0] = x[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 t = x.two(i);
            f[i] = t.x;
            f[i + 1] = t.y;
        }
    }
}
template <typename T, int V> __device__ __forceinline__ void narrow(Vec<T, V> &x, const float (&f)[V]) {
    if constexpr (V == 1) {
        x.v[0] = from_f32<T>(f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) x.put(i, make_float2(f[i], f[i + 1]));
    }
}

// A CTA of kThreads takes pieces of kPiece tokens of CH channels (128 bytes of a row) in turn, the next
// pieces' rows on their way into shared memory meanwhile.  A thread walks a run of kRun tokens of V
// channels with its last W inputs in registers.
//
// ODD: rows of 16-bit elements that begin on no 4-byte boundary all the same.  They are copied in the
// 4-byte words that they lie in (a word never ends outside the allocation that one of its bytes is in)
// and are shifted by an element when they are read: element by element, copies and their
// addresses would be most of the kernel.
constexpr int kThreads = 128, V = 4, kPiece = kConvPiece;

template <typename T, bool ODD> struct Shape {
    static constexpr int LANES = 128 / (V * sizeof(T)), CH = LANES * V, kRuns = kThreads / LANES;
    static constexpr int kRun = kPiece / kRuns;
    static constexpr int kRow = ODD ? 136 : 128;  // bytes of a row in shared memory
};

// Whether a row's first element lies in the middle of a 4-byte word.
template <typename T> __device__ __forceinline__ int shifted(const void *base, long long element) {
    return sizeof(T) == 2 ? (int)(((uintptr_t)base >> 1) + (unsigned long long)element) & 1 : 0;
}

// A thread's channels out of a row in shared memory; `bits`: 16 where the row is shifted.
template <typename T, bool ODD> __device__ __forceinline__ Vec<T, V> take(const char *at, int bits) {
    if constexpr (!ODD) {
        return *(const Vec<T, V> *)at;
    } else {
        const uint2 lo = *(const uint2 *)at;
        const uint32_t hi = *(const uint32_t *)(at + 8);
        Vec<T, V> x;
        *(uint2 *)&x = make_uint2(__funnelshift_r(lo.x, lo.y, bits), __funnelshift_r(lo.y, hi, bits));
        return x;
    }
}

__device__ __forceinline__ void copy4(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// Rows [pos, end) of a sequence into rows from `to` on, neighbouring threads neighbouring words of `unit`
// bytes; zeros outside the sequence and behind the last channel.  (A thread's rows are four apart, or
// a multiple, so that all of them are shifted alike.)
template <typename T, bool ODD>
__device__ __forceinline__ void fetch_rows(char *to, const ConvArgs &a, const Piece &p, const void *base,
                                           long long stride, int pos, int end, int c0, int unit) {
    constexpr int kRow = Shape<T, ODD>::kRow, E = sizeof(T);
    const int shift = ODD || unit == 4 ? 5 : unit == 8 ? 4 : 3;  // words of a row: 1 << shift
    if (ODD) unit = 4;
    const int word = threadIdx.x & ((1 << shift) - 1), row = threadIdx.x >> shift, step = kThreads >> shift;
    const long long first = (p.row0 + pos + row) * stride + c0;
    const int s = ODD ? 2 * shifted<T>(base, first) : 0;
    const int left = (a.D - c0) * E + s;                          // bytes of the row from its first word on
    const int most = min(unit, left - word * unit), tail = min(4, left - 128);  // of this word, of the 33rd
    const char *at = (const char *)base + first * E - s + word * unit;
    // an address for copies of nothing: the rows' own, which a batch of no tokens may not have
    const char *any = base ? (const char *)((uintptr_t)base & ~(uintptr_t)3)
                           : (const char *)((uintptr_t)a.weight & ~(uintptr_t)15);
    uint32_t d = (uint32_t)__cvta_generic_to_shared(to) + row * kRow + word * unit;
    const long long ahead = step * stride * E;
    const bool last = ODD && s && word == 0;
    auto ok = [&](int x) {
        return x >= 0 && x < p.total && in_bounds(a.dbg, (size_t)(p.row0 + x), (size_t)a.tok.rows(), DBG_LOAD);
    };
    auto each = [&](auto copy) {
        int x = pos + row;
        if (pos >= 0 && end <= p.total && most == unit && (!last || tail == 4) && ok(end - 1)) {
#pragma unroll 4
            for (; x < end; x += step, at += ahead, d += step * kRow) {
                copy(d, at, unit);
                if (last) copy4(d + 128, at + 128, 4);
            }
        } else {
            for (; x < end; x += step, at += ahead, d += step * kRow) {
                const bool in = ok(x) && most > 0;
                copy(d, in ? at : any, in ? most : 0);
                if (last) {
                    const bool more = ok(x) && tail > 0;
                    copy4(d + 128, more ? at + 128 : any, more ? tail : 0);
                }
            }
        }
    };
    if (!ODD && unit == 16)
        each([](uint32_t d, const char *f, int n) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(f), "r"(n) : "memory");
        });
    else if (!ODD && unit == 8)
        each([](uint32_t d, const char *f, int n) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(f), "r"(n) : "memory");
        });
    else
        each([](uint32_t d, const char *f, int n) { copy4(d, f, n); });
}
// x from W - 1 rows in front of a piece (the inputs in front of the sequence among them) to `end`.
template <typename T, int W, bool ODD>
__device__ __forceinline__ void fetch_inputs(char *to, const ConvArgs &a, const Piece &p, int end, int c0, int unit) {
    using S = Shape<T, ODD>;
    const int front = p.begin == 0 && a.initial ? W - 1 : 0;
    fetch_rows<T, ODD>(to + front * S::kRow, a, p, a.x, a.x_stride, p.begin - (W - 1) + front, end, c0, unit);
    for (int i = threadIdx.x; i < front * S::CH; i += kThreads) {
        const int r = i / S::CH, e = i % S::CH;
        const size_t row = (size_t)p.seq * (W - 1) + r;
        const bool ok = c0 + e < a.D && in_bounds(a.dbg, row, (size_t)a.tok.num_seqs * (W - 1), DBG_LOAD);
        const int s = ODD ? shifted<T>(a.x, (p.row0 + r - (W - 1)) * a.x_stride + c0) : 0;
        ((T *)(to + r * S::kRow))[s + e] = ok ? ((const T *)a.initial)[row * a.D + c0 + e] : from_f32<T>(0.f);
    }
}
// Rows of a piece from shared memory [kPiece][CH], where a thread's channels are on no boundary of their
// own in the tensor: a warp a row (all of its rows are shifted alike), words where they are whole.
template <typename T, int CH>
__device__ __forceinline__ void leave_rows(const T (*from)[CH], const ConvArgs &a, const Piece &p, void *base,
                                           long long stride, int c0) {
    constexpr int kStep = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, left = min(CH, a.D - c0);
    if (!in_bounds(a.dbg, (size_t)(p.row0 + p.begin + p.len - 1), (size_t)a.tok.rows(), DBG_STORE)) return;
    const long long first = (p.row0 + p.begin + warp) * stride + c0;
    T *to = (T *)base + first;
    if constexpr (sizeof(T) == 4) {
        if (lane >= left) return;
#pragma unroll 4
        for (int r = warp; r < p.len; r += kStep, to += kStep * stride) to[lane] = from[r][lane];
    } else {
        const int s = shifted<T>(base, first), e = 2 * lane - s;  // this lane's word: channels e, e + 1
        const bool whole = e >= 0 && e + 1 < left, lo = e >= 0 && e < left, hi = e + 1 < left;
        const bool last = s && lane == 0 && CH <= left;  // the row's last channel is in a word of its own
        uint16_t *t = (uint16_t *)to + e;
#pragma unroll 4
        for (int r = warp; r < p.len; r += kStep, t += kStep * stride) {
            const uint16_t *f = (const uint16_t *)from[r] + e;
            if (whole) {
                *(uint32_t *)t = s ? f[0] | (uint32_t)f[1] << 16 : *(const uint32_t *)f;
            } else {
                if (lo) t[0] = f[0];
                if (hi) t[1] = f[1];
            }
            if (last) t[CH] = f[CH];  // (e = -1)
        }
    }
}
// CTAs with so much shared memory that a multiprocessor holds, at most `most`.
inline long long resident(int bytes, int most) {
    const int n = 228 * 1024 / (bytes + 1024);
    return n < most ? n : most;
}

template <int W, int CH>
__device__ __forceinline__ void load_params(const ConvArgs &a, int c0, float (*w)[CH]) {
    for (int i = threadIdx.x; i < CH; i += kThreads) {
        const bool in = c0 + i < a.D && in_bounds(a.dbg, (size_t)(c0 + i), (size_t)a.D, DBG_LOAD);
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = in ? param(a.weight, a.wdtype, (size_t)(c0 + i) * W + j, 0.f) : 0.f;
        w[W][i] = in ? param(a.bias, a.wdtype, c0 + i, 0.f) : 0.f;
    }
}

}  // namespace conv
}  // namespace kda
