// Short causal convolution, forward, and its single-token form.
//
// Bound by memory: x is read and y written once.  A warp takes 8 tokens of 32 V channels, V those
// of an 8-byte load (16 in FP32); every row that they need (8 and the W - 1 in front) is asked for before
// the first is used, so that a multiprocessor has some 90 KB on their way in 32 warps; the rows that two
// warps both read come out of the cache.  (With 16-byte loads of 16-bit types a thread needs 149
// registers, and one CTA a multiprocessor is left: 644 us at B=8 T=4096 D=6144.)
#include "kda_conv.cuh"

namespace kda {
namespace conv {
namespace {

constexpr int kRun = 8, kWarps = 8, kPiece = kRun * kWarps;

template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * kWarps, V == 1 ? 6 : 3) kda_conv_fwd_kernel(const ConvArgs a, int blocks) {
    wait_for_previous();
    __shared__ __align__(16) float w[W + 1][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (int)(blockIdx.x % (unsigned)blocks) * 32 * V, c = c0 + lane * V;
    const Piece p = find_piece(a.tok, blockIdx.x / (unsigned)blocks, kPiece);
    if (p.len < 0) return;
    load_params<V, W>(a, c0, w, 32 * kWarps);
    const int t0 = p.begin + warp * kRun, n = min(kRun, p.begin + p.len - t0);
    const bool in = c < a.D;
    Vec<T, V> x[kRun + W - 1];
    if (in && n > 0) {
        if (t0 >= W - 1 && t0 + kRun <= p.total &&
            dbg_ok(a.dbg, (size_t)(p.row0 + t0 + kRun - 1), (size_t)a.tok.rows(), DBG_LOAD)) {
            const T *at = (const T *)a.x + (p.row0 + t0 - (W - 1)) * a.x_stride + c;
#pragma unroll
            for (int i = 0; i < kRun + W - 1; ++i) {
                x[i] = *reinterpret_cast<const Vec<T, V> *>(at);
                at += a.x_stride;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kRun + W - 1; ++i) x[i] = input<T, V>(a, p, t0 + i - (W - 1), W, c);
        }
    }
    __syncthreads();
    if (!in) return;
    if (n > 0) {
#pragma unroll
        for (int t = 0; t < kRun; ++t) {
            float acc[V];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = w[W][lane * V + i];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float xv[V], wv[V];
                widen(xv, x[t + j]);
#pragma unroll
                for (int i = 0; i < V; ++i) wv[i] = w[j][lane * V + i];
                vfma(acc, xv, wv);
            }
            const long long row = p.row0 + t0 + t;
            if (t < n && dbg_ok(a.dbg, (size_t)row, (size_t)a.tok.rows(), DBG_STORE)) {
                Vec<T, V> y;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    y.v[i] = from_f32<T>(a.act == ACT_SILU ? acc[i] * sigmoid(acc[i]) : acc[i]);
                *reinterpret_cast<Vec<T, V> *>((T *)a.y + row * a.y_stride + c) = y;
            }
        }
    }
    if (a.final && p.begin + p.len == p.total && warp < W - 1) {  // the sequence's last inputs
        const size_t row = (size_t)p.seq * (W - 1) + warp;
        if (dbg_ok(a.dbg, row, (size_t)a.tok.num_seqs * (W - 1), DBG_STORE))
            *reinterpret_cast<Vec<T, V> *>((T *)a.final + row * a.D + c) =
                input<T, V>(a, p, p.total - (W - 1) + warp, W, c);
    }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(256) kda_conv_step_kernel(const ConvArgs a) {
    wait_for_previous();
    const int c = (int)(blockIdx.x * blockDim.x + threadIdx.x) * V, n = blockIdx.y;
    if (c >= a.D) return;
    long long slot = a.state_indices ? a.state_indices[n] : n;
    const bool none = slot < 0 || slot >= a.num_states;  // no request here: y is zero
    Vec<T, V> y, x[W];
    y.clear();
    if (!none && dbg_ok(a.dbg, (size_t)n, (size_t)a.N, DBG_LOAD)) {
        T *st = (T *)a.state + (size_t)slot * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) x[j] = *reinterpret_cast<const Vec<T, V> *>(st + (size_t)j * a.D);
        x[W - 1] = *reinterpret_cast<const Vec<T, V> *>((const T *)a.x + n * a.x_stride + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float acc = param(a.bias, a.wdtype, c + i, 0.f);
#pragma unroll
            for (int j = 0; j < W; ++j)
                acc = fmaf(x[j][i], param(a.weight, a.wdtype, (size_t)(c + i) * W + j, 0.f), acc);
            y.v[i] = from_f32<T>(a.act == ACT_SILU ? acc * sigmoid(acc) : acc);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<Vec<T, V> *>(st + (size_t)j * a.D) = x[j + 1];
    }
    if (dbg_ok(a.dbg, (size_t)n, (size_t)a.N, DBG_STORE))
        *reinterpret_cast<Vec<T, V> *>((T *)a.y + n * a.y_stride + c) = y;
}

template <typename T, int V, int W> cudaError_t forward(const ConvArgs &a, cudaStream_t stream) {
    const int blocks = (a.D + 32 * V - 1) / (32 * V);
    return launch_early(kda_conv_fwd_kernel<T, V, W>, (unsigned)(a.tok.pieces(kPiece) * blocks),
                        32 * kWarps, 0, stream, a, blocks);
}
template <typename T, int V> cudaError_t forward(const ConvArgs &a, cudaStream_t stream) {
    return a.W == 4 ? forward<T, V, 4>(a, stream) : a.W == 3 ? forward<T, V, 3>(a, stream)
                                                             : forward<T, V, 2>(a, stream);
}
template <typename T> cudaError_t forward(const ConvArgs &a, cudaStream_t stream) {
    return vec_ok(a, 4) ? forward<T, 4>(a, stream) : forward<T, 1>(a, stream);
}

template <typename T, int V, int W> cudaError_t step(const ConvArgs &a, cudaStream_t stream) {
    // 64 threads a block: a few requests are spread over more multiprocessors
    const unsigned blocks = (unsigned)((a.D + 64 * V - 1) / (64 * V));
    return launch_early(kda_conv_step_kernel<T, V, W>, dim3(blocks, (unsigned)a.N), 64, 0, stream, a);
}
template <typename T, int V> cudaError_t step(const ConvArgs &a, cudaStream_t stream) {
    return a.W == 4 ? step<T, V, 4>(a, stream) : a.W == 3 ? step<T, V, 3>(a, stream)
                                                          : step<T, V, 2>(a, stream);
}
template <typename T> cudaError_t step(const ConvArgs &a, cudaStream_t stream) {
    constexpr int V = 8 / sizeof(T);
    return vec_ok(a, V) && aligned(a.state, 8) ? step<T, V>(a, stream) : step<T, 1>(a, stream);
}

}  // namespace
}  // namespace conv

cudaError_t launch_conv_fwd(const ConvArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return conv::forward<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return conv::forward<__half>(a, stream);
    return conv::forward<float>(a, stream);
}

cudaError_t launch_conv_step(const ConvArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return conv::step<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return conv::step<__half>(a, stream);
    return conv::step<float>(a, stream);
}

}  // namespace kda
