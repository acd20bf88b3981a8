// Short causal convolution, forward, and its single-token form.
//
// Bound by memory: x is read and y written once.  Rows come through shared memory, two pieces ahead
// (kda_conv.cuh): 140 us at B=8 T=4096 D=6144 W=4 bf16 with silu, 5.7 TB/s, 85% of a copy's rate.  (Loads
// into registers eight tokens ahead: 188 us, with a third of the instructions moving and addressing
// them.  Stores marked as not to be kept in L2: 148.)  9467 tokens of 1111 fp16 channels
// take 28.7 us (x's rows, a slice's, begin on 4-byte boundaries there, y's on none), of 1112 15.0: what odd
// rows add is copies of 4-byte words and y's way out through shared memory, at 38% of the issue slots and 9%
// of memory's rate, four warps a scheduler that wait in turn.
//
// Single tokens (kda_conv_step_kernel): a thread has four channels of a request, the last inputs and
// the token in registers; a few requests are the latency of one launch (2 us beside the host's 4).
#include <type_traits>

#include "kda_conv.cuh"

namespace kda {
namespace conv {
namespace {

constexpr int kStages = 3;

template <typename T, int W, bool ODD> struct Smem {
    using S = Shape<T, ODD>;
    char x[kStages][kPiece + W - 1][S::kRow];
    float w[W + 1][S::CH];
    T y[kPiece][S::CH];  // only where y's rows are on no boundary of V elements
};

template <typename T, int W, bool ODD>
__global__ void __launch_bounds__(kThreads, 4)
    kda_conv_fwd_kernel(const ConvArgs a, long long pieces, int unit_x, int unit_y) {
    wait_for_previous();
    using S = Shape<T, ODD>;
    using M = Smem<T, W, ODD>;
    extern __shared__ __align__(16) char smem[];
    M &s = *reinterpret_cast<M *>(smem);
    const int lane = threadIdx.x % S::LANES, run = threadIdx.x / S::LANES;
    const int c0 = blockIdx.x * S::CH, c = c0 + lane * V, left = a.D - c;
    const bool wide = unit_y >= (int)(V * sizeof(T));
    auto piece = [&](long long at) {
        Piece p;
        p.len = -1;
        return at < pieces ? find_piece(a.tok, at, kPiece) : p;
    };
    auto fetch = [&](const Piece &p, int stage) {
        if (p.len >= 0) fetch_inputs<T, W, ODD>(s.x[stage][0], a, p, p.begin + p.len, c0, unit_x);
        cp_async_commit();
    };
    load_params<W>(a, c0, s.w);
    Piece p = piece(blockIdx.y), p1 = piece(blockIdx.y + (long long)gridDim.y);
    fetch(p, 0);
    fetch(p1, 1);
    __syncthreads();
    float w[W][V], bias[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = s.w[j][lane * V + e];
        bias[e] = s.w[W][lane * V + e];
    }
    int b = 0;
    for (long long at = blockIdx.y; at < pieces; at += gridDim.y) {
        const Piece p2 = piece(at + 2LL * gridDim.y);
        fetch(p2, b > 0 ? b - 1 : kStages - 1);
        cp_async_wait_newest<2>();
        __syncthreads();
        const int r0 = run * S::kRun, n = p.len - r0;
        if (n > 0 && left > 0) {
            const char *xs = s.x[b][r0] + lane * V * sizeof(T);
            int bits[2] = {};  // of rows an even and an odd number behind the run's first one
            if (ODD) {
                const long long e = (p.row0 + p.begin + r0 - (W - 1)) * a.x_stride + c0;
                bits[0] = 16 * shifted<T>(a.x, e);
                bits[1] = 16 * shifted<T>(a.x, e + a.x_stride);
            }
            T *out = wide ? (T *)a.y + (p.row0 + p.begin + r0) * a.y_stride + c : &s.y[r0][lane * V];
            const long long step = wide ? a.y_stride : S::CH;
            auto walk = [&](auto whole) {
                float x[W][V];  // the input of token i is at i % W
#pragma unroll
                for (int j = 0; j < W - 1; ++j) widen(x[(j + 1) % W], take<T, ODD>(xs + j * S::kRow, bits[j & 1]));
#pragma unroll
                for (int i = 0; i < S::kRun; ++i) {
                    if (!whole && i >= n) break;
                    widen(x[i % W], take<T, ODD>(xs + (i + W - 1) * S::kRow, bits[(i + W - 1) & 1]));
                    float acc[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = bias[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) vfma(acc, x[(i + 1 + j) % W], w[j]);
                    if (a.act == ACT_SILU) {
#pragma unroll
                        for (int e = 0; e < V; ++e) acc[e] *= sigmoid(acc[e]);
                    }
                    Vec<T, V> y;
                    narrow(y, acc);
                    if (in_bounds(a.dbg, (size_t)(p.row0 + p.begin + r0 + i), (size_t)a.tok.rows(), DBG_STORE))
                        *(Vec<T, V> *)out = y;
                    out += step;
                }
            };
            if (n >= S::kRun)
                walk(std::true_type());
            else
                walk(std::false_type());
        }
        if (a.final && p.len >= 0 && p.begin + p.len == p.total) {  // the sequence's last inputs
            for (int i = threadIdx.x; i < (W - 1) * S::CH; i += kThreads) {
                const int r = i / S::CH, e = i % S::CH;
                const size_t row = (size_t)p.seq * (W - 1) + r;
                const long long at = (p.row0 + p.total - (W - 1) + r) * a.x_stride + c0;
                if (c0 + e < a.D && in_bounds(a.dbg, row, (size_t)a.tok.num_seqs * (W - 1), DBG_STORE))
                    ((T *)a.final)[row * a.D + c0 + e] =
                        ((const T *)s.x[b][p.len + r])[(ODD ? shifted<T>(a.x, at) : 0) + e];
            }
        }
        __syncthreads();
        if (!wide && p.len > 0) leave_rows<T, S::CH>(s.y, a, p, a.y, a.y_stride, c0);
        p = p1;
        p1 = p2;
        b = b + 1 < kStages ? b + 1 : 0;
    }
    cp_async_wait_newest<0>();
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
    if (!none && in_bounds(a.dbg, (size_t)n, (size_t)a.N, DBG_LOAD) &&
        in_bounds(a.dbg, ((size_t)(slot + 1) * (W - 1) - 1) * a.D + c + V - 1, (size_t)a.num_states * (W - 1) * a.D, DBG_STORE)) {
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
    if (in_bounds(a.dbg, (size_t)n, (size_t)a.N, DBG_STORE))
        *reinterpret_cast<Vec<T, V> *>((T *)a.y + n * a.y_stride + c) = y;
}

template <typename T, int W, bool ODD>
cudaError_t forward(const ConvArgs &a, int unit_x, int unit_y, cudaStream_t stream) {
    using M = Smem<T, W, ODD>;
    const long long pieces = a.tok.pieces(kPiece);
    const unsigned blocks = (unsigned)((a.D + M::S::CH - 1) / M::S::CH);
    constexpr int kBytes = sizeof(M);
    const int bytes = unit_y >= (int)(V * sizeof(T)) ? kBytes - (int)sizeof(M::y) : kBytes;
    const long long wave = resident(bytes, 4) * kSMs / blocks, most = wave > 1 ? wave : 1;
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = smem_limit_once(kda_conv_fwd_kernel<T, W, ODD>, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    return launch_early(kda_conv_fwd_kernel<T, W, ODD>, dim3(blocks, (unsigned)(pieces < most ? pieces : most)),
                        kThreads, bytes, stream, a, pieces, unit_x, unit_y);
}
template <typename T, int W> cudaError_t forward(const ConvArgs &a, cudaStream_t stream) {
    rows::Boundary x(sizeof(T), 16), y(sizeof(T), a.D);  // (the last channels of a row may be part of a word)
    x.add(a.x, a.x_stride);
    y.add(a.y, a.y_stride);
    if constexpr (sizeof(T) == 2)
        if (x.unit < 4) return forward<T, W, true>(a, x.unit, y.unit, stream);
    return forward<T, W, false>(a, x.unit, y.unit, stream);
}
template <typename T> cudaError_t forward(const ConvArgs &a, cudaStream_t stream) {
    return a.W == 4 ? forward<T, 4>(a, stream) : a.W == 3 ? forward<T, 3>(a, stream) : forward<T, 2>(a, stream);
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
    const bool wide = a.D % V == 0 && aligned(a.x, 8) && aligned(a.y, 8) && aligned(a.state, 8) &&
                      a.x_stride % V == 0 && a.y_stride % V == 0;
    return wide ? step<T, V>(a, stream) : step<T, 1>(a, stream);
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
