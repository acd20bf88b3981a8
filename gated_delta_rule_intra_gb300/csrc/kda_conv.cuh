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
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = x[i];
}

// The input at position `pos` of a sequence, in front of it and behind it too.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> input(const ConvArgs &a, const Piece &p, int pos, int W, int c) {
    Vec<T, V> x;
    if (pos >= p.total || (pos < 0 && !a.initial)) {
        x.clear();
        return x;
    }
    const T *at;
    if (pos >= 0) {
        const long long row = p.row0 + pos;
        at = dbg_ok(a.dbg, (size_t)row, (size_t)a.tok.rows(), DBG_LOAD)
                 ? (const T *)a.x + row * a.x_stride + c : (const T *)a.x + c;
    } else {
        const size_t row = (size_t)p.seq * (W - 1) + (pos + W - 1);
        at = (const T *)a.initial +
             (dbg_ok(a.dbg, row, (size_t)a.tok.num_seqs * (W - 1), DBG_LOAD) ? row * a.D + c : c);
    }
    return *reinterpret_cast<const Vec<T, V> *>(at);
}

// The block's weights and biases as [W + 1][32 V] floats.
template <int V, int W>
__device__ __forceinline__ void load_params(const ConvArgs &a, int c0, float (*w)[32 * V], int threads) {
    for (int i = threadIdx.x; i < 32 * V; i += threads) {
        const bool in = c0 + i < a.D;
#pragma unroll
        for (int j = 0; j < W; ++j)
            w[j][i] = in ? param(a.weight, a.wdtype, (size_t)(c0 + i) * W + j, 0.f) : 0.f;
        w[W][i] = in ? param(a.bias, a.wdtype, c0 + i, 0.f) : 0.f;
    }
}

// Accesses of v elements need rows on such boundaries.
inline bool vec_ok(const ConvArgs &a, int v) {
    const size_t b = (size_t)v * esize(a.dtype);
    auto ok = [&](const void *p, long long stride) { return aligned(p, b) && stride % v == 0; };
    return a.D % v == 0 && ok(a.x, a.x_stride) && ok(a.initial, v) && ok(a.final, v) && ok(a.y, a.y_stride);
}

}  // namespace conv
}  // namespace kda
