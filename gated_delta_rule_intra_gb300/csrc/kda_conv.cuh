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
// pieces' rows on their way into shared memory meanwhile, whatever their alignment.  A thread walks
// a run of kRun tokens of V channels with its last W inputs in registers.
constexpr int kThreads = 128, V = 4, kPiece = kConvPiece;

template <typename T> struct Shape {
    static constexpr int LANES = 128 / (V * sizeof(T)), CH = LANES * V, kRuns = kThreads / LANES;
    static constexpr int kRun = kPiece / kRuns;
    static constexpr int kChunks = CH / 8, kRowStep = kThreads / kChunks;
};

// Rows [pos, end) of a sequence into rows of shared memory, this thread's kRowStep apart and its eight
// channels of them; zeros outside the sequence.
template <typename T>
__device__ __forceinline__ void fetch_rows(T (*to)[Shape<T>::CH], const ConvArgs &a, const Piece &p, const void *base,
                                           long long stride, int pos, int end, int c, int left, int unit) {
    constexpr int kStep = Shape<T>::kRowStep;
    const T *at = (const T *)base + (p.row0 + pos) * stride + c;
    for (; pos < end; pos += kStep, at += kStep * stride, to += kStep) {
        const bool ok = pos >= 0 && pos < p.total &&
                        dbg_ok(a.dbg, (size_t)(p.row0 + pos), (size_t)a.tok.rows(), DBG_LOAD);
        fetch_chunk<T>((Vec<T, 8> *)to[0], base, at, left, ok, unit);
    }
}
// x from W - 1 rows in front of a piece (the inputs in front of the sequence among them) on.
template <typename T, int W>
__device__ __forceinline__ void fetch_inputs(T (*to)[Shape<T>::CH], const ConvArgs &a, const Piece &p, int end, int c0,
                                             int unit) {
    const int r = threadIdx.x / Shape<T>::kChunks, e = threadIdx.x % Shape<T>::kChunks * 8, c = c0 + e;
    const int pos = p.begin - (W - 1) + r;
    T(*mine)[Shape<T>::CH] = (T(*)[Shape<T>::CH])&to[r][e];
    fetch_rows<T>(mine, a, p, a.x, a.x_stride, pos, end, c, a.D - c, unit);
    if (pos < 0 && a.initial) {
        const long long row = (long long)p.seq * (W - 1) + pos + W - 1;
        fetch_chunk<T>((Vec<T, 8> *)mine, a.initial, (const T *)a.initial + row * a.D + c, a.D - c,
                       dbg_ok(a.dbg, (size_t)row, (size_t)a.tok.num_seqs * (W - 1), DBG_LOAD), unit);
    }
}
// A thread's channels of a row; `wide`: all of them, on such a boundary.
template <typename T>
__device__ __forceinline__ void store_channels(T *to, const Vec<T, V> &x, int left, bool wide) {
    if (wide) {
        *reinterpret_cast<Vec<T, V> *>(to) = x;
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < left) to[e] = x.v[e];
    }
}
template <int W, int CH>
__device__ __forceinline__ void load_params(const ConvArgs &a, int c0, float (*w)[CH]) {
    for (int i = threadIdx.x; i < CH; i += kThreads) {
        const bool in = c0 + i < a.D;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = in ? param(a.weight, a.wdtype, (size_t)(c0 + i) * W + j, 0.f) : 0.f;
        w[W][i] = in ? param(a.bias, a.wdtype, c0 + i, 0.f) : 0.f;
    }
}

}  // namespace conv
}  // namespace kda
