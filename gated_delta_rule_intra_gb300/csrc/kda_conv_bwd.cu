// Short causal convolution, backward: with g = dy act'(pre), pre computed again from x,
//   dx[t] = sum_j weight[j] g[t + W - 1 - j],
//   dweight[j] = sum over tokens of g[t] x[t - W + 1 + j],  dbias = sum over tokens of g.
// The final state's gradient is that of the sequence's last inputs and is added to theirs.
//
// Bound by memory (x and dy read, dx written once).  A warp walks a run of 16 tokens of 32 V
// channels with the last W inputs and the last W values of g in registers, and W - 1 tokens more
// whose g its last inputs need; the next four tokens' rows are on their way.  A resident CTA takes
// pieces of 128 tokens of its channels in turn and keeps the parameters' sums in registers; the
// CTAs' sums are added up in a fixed order by a second kernel.
#include "kda_conv.cuh"

namespace kda {
namespace conv {
namespace {

constexpr int kRun = 16, kWarps = 8, kPiece = kRun * kWarps, kAhead = 4;
static_assert(kPiece == kConvPiece, "");

template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * kWarps, 2) kda_conv_bwd_kernel(const ConvArgs a, long long pieces) {
    wait_for_previous();
    __shared__ __align__(16) float w[W + 1][32 * V];
    __shared__ float red[kWarps][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.x * 32 * V, c = c0 + lane * V;
    const bool in = c < a.D;
    load_params<V, W>(a, c0, w, 32 * kWarps);
    __syncthreads();
    float wv[W][V], bias[V], dw[W][V] = {}, db[V] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) wv[j][i] = w[j][lane * V + i];
        bias[i] = w[W][lane * V + i];
    }
    for (long long at = blockIdx.y; at < pieces; at += gridDim.y) {
        const Piece p = find_piece(a.tok, at, kPiece);
        if (p.len <= 0) continue;
        const int t0 = p.begin + warp * kRun, n = min(kRun, p.begin + p.len - t0);
        if (!in || n <= 0) continue;
        const int steps = n + W - 1;
        auto grad = [&](int pos) {  // dy at a position
            Vec<T, V> x;
            x.clear();
            const long long row = p.row0 + pos;
            if (pos < p.total && dbg_ok(a.dbg, (size_t)row, (size_t)a.tok.rows(), DBG_LOAD))
                x = *reinterpret_cast<const Vec<T, V> *>((const T *)a.dy + row * a.dy_stride + c);
            return x;
        };
        Vec<T, V> nx[kAhead], ny[kAhead];
        float xw[W][V] = {}, gw[W][V] = {};
#pragma unroll
        for (int j = 0; j < W - 1; ++j) widen(xw[j + 1], input<T, V>(a, p, t0 - (W - 1) + j, W, c));
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            nx[k] = input<T, V>(a, p, t0 + k, W, c);
            ny[k] = grad(t0 + k);
        }
        for (int base = 0; base < steps; base += kAhead) {
            Vec<T, V> x[kAhead], dy[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                x[k] = nx[k];
                dy[k] = ny[k];
            }
            if (base + kAhead < steps) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    nx[k] = input<T, V>(a, p, t0 + base + kAhead + k, W, c);
                    ny[k] = grad(t0 + base + kAhead + k);
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = base + k;
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        xw[j][e] = xw[j + 1][e];
                        gw[j][e] = gw[j + 1][e];
                    }
                widen(xw[W - 1], x[k]);
                float g[V];
                widen(g, dy[k]);
                if (a.act == ACT_SILU) {
                    float pre[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) pre[e] = bias[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) vfma(pre, xw[j], wv[j]);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        // (a position behind the sequence has dy = 0 and x = 0)
                        const float s = sigmoid(pre[e]);
                        g[e] = t0 + i < p.total ? g[e] * silu_slope(pre[e], s) : 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < V; ++e) gw[W - 1][e] = g[e];
                if (i < n) {
#pragma unroll
                    for (int j = 0; j < W; ++j) vfma(dw[j], g, xw[j]);
#pragma unroll
                    for (int e = 0; e < V; ++e) db[e] += g[e];
                }
                if (i >= W - 1 && i < steps) {
                    float dx[V] = {};
#pragma unroll
                    for (int j = 0; j < W; ++j) vfma(dx, wv[j], gw[W - 1 - j]);
                    const int pos = t0 + i - (W - 1);
                    const int last = pos - (p.total - (W - 1));
                    if (a.d_final && last >= 0) {
                        const size_t row = (size_t)p.seq * (W - 1) + last;
                        if (dbg_ok(a.dbg, row, (size_t)a.tok.num_seqs * (W - 1), DBG_LOAD)) {
                            const auto f = *reinterpret_cast<const Vec<T, V> *>((const T *)a.d_final + row * a.D + c);
#pragma unroll
                            for (int e = 0; e < V; ++e) dx[e] += f[e];
                        }
                    }
                    Vec<T, V> out;
#pragma unroll
                    for (int e = 0; e < V; ++e) out.v[e] = from_f32<T>(dx[e]);
                    const long long row = p.row0 + pos;
                    if (dbg_ok(a.dbg, (size_t)row, (size_t)a.tok.rows(), DBG_STORE))
                        *reinterpret_cast<Vec<T, V> *>((T *)a.dx + row * a.dx_stride + c) = out;
                }
            }
        }
    }
    if (!a.dweight) return;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) red[warp][lane * V + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * V; i += 32 * kWarps) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) s += red[k][i];
            if (c0 + i < a.D && dbg_ok(a.dbg, blockIdx.y, (size_t)a.partials, DBG_STORE))
                a.partial[((size_t)blockIdx.y * (W + 1) + j) * a.D + c0 + i] = s;
        }
    }
}

// The parameters' gradients: sums of `partial`'s rows, in order.
__global__ void __launch_bounds__(256) kda_conv_sum_kernel(const ConvArgs a) {
    wait_for_previous();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int j = (int)(i / a.D), c = (int)(i % a.D);
    if (j > a.W) return;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < a.partials; ++k) s += a.partial[((size_t)k * (a.W + 1) + j) * a.D + c];
    if (j < a.W)
        a.dweight[(size_t)c * a.W + j] = s;
    else
        a.dbias[c] = s;
}

// Gradients of the inputs in front of each sequence: its first W - 1 values of g again.
template <typename T> __global__ void __launch_bounds__(256) kda_conv_initial_kernel(const ConvArgs a) {
    wait_for_previous();
    const int c = blockIdx.x * 256 + threadIdx.x, n = blockIdx.y, W = a.W;
    if (c >= a.D) return;
    Piece p;
    p.seq = n;
    if (a.tok.cu_seqlens) {
        auto token = [&](int v) { return v < 0 ? 0 : v > a.tok.T ? a.tok.T : v; };
        const int lo = token(a.tok.cu_seqlens[n]), hi = token(a.tok.cu_seqlens[n + 1]);
        p.row0 = lo;
        p.total = hi > lo ? hi - lo : 0;
    } else {
        p.row0 = (long long)n * a.tok.T;
        p.total = a.tok.T;
    }
    float d[3] = {};
    for (int t = 0; t < W - 1 && t < p.total; ++t) {
        float g = as_f32(((const T *)a.dy)[(p.row0 + t) * a.dy_stride + c]);
        if (a.act == ACT_SILU) {
            float pre = param(a.bias, a.wdtype, c, 0.f);
            for (int j = 0; j < W; ++j)
                pre = fmaf(input<T, 1>(a, p, t - (W - 1) + j, W, c)[0],
                           param(a.weight, a.wdtype, (size_t)c * W + j, 0.f), pre);
            g *= silu_slope(pre, sigmoid(pre));
        }
        for (int r = t; r < W - 1; ++r)  // input r - (W - 1) is token t's tap r - t
            d[r] = fmaf(g, param(a.weight, a.wdtype, (size_t)c * W + r - t, 0.f), d[r]);
    }
    for (int r = 0; r < W - 1; ++r) {
        const int last = r - p.total;  // where it is still among the last inputs
        if (a.d_final && last >= 0)
            d[r] += as_f32(((const T *)a.d_final)[((size_t)n * (W - 1) + last) * a.D + c]);
        if (dbg_ok(a.dbg, (size_t)n, (size_t)a.tok.num_seqs, DBG_STORE))
            ((T *)a.d_initial)[((size_t)n * (W - 1) + r) * a.D + c] = from_f32<T>(d[r]);
    }
}

template <typename T, int V, int W> cudaError_t backward(const ConvArgs &a, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((a.D + 32 * V - 1) / (32 * V));
    const long long pieces = a.tok.pieces(kPiece);
    ConvArgs b = a;  // as many rows of sums as CTAs
    const long long most = (2 * kSMs) / (long long)blocks > 1 ? (2 * kSMs) / (long long)blocks : 1;
    const long long rows = pieces < most ? pieces : most;
    if (rows < b.partials || !a.dweight) b.partials = (int)rows;
    cudaError_t e = launch_early(kda_conv_bwd_kernel<T, V, W>, dim3(blocks, (unsigned)b.partials),
                                 32 * kWarps, 0, stream, b, pieces);
    if (e != cudaSuccess || !a.dweight) return e;
    return launch_early(kda_conv_sum_kernel, (unsigned)(((long long)(W + 1) * a.D + 255) / 256), 256, 0, stream, b);
}
template <typename T, int V> cudaError_t backward(const ConvArgs &a, cudaStream_t stream) {
    return a.W == 4 ? backward<T, V, 4>(a, stream) : a.W == 3 ? backward<T, V, 3>(a, stream)
                                                              : backward<T, V, 2>(a, stream);
}
template <typename T> cudaError_t backward(const ConvArgs &a, cudaStream_t stream) {
    if (a.d_initial) {
        const cudaError_t e = launch_early(kda_conv_initial_kernel<T>,
                                           dim3((unsigned)((a.D + 255) / 256), (unsigned)a.tok.num_seqs),
                                           256, 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return vec_ok(a, 4, true) ? backward<T, 4>(a, stream) : backward<T, 1>(a, stream);
}

}  // namespace
}  // namespace conv

// CTAs of a block of channels, each with a row of sums: one wave of them, of either block width.
int conv_partials(long long pieces, int D) {
    const long long blocks = (D + 127) / 128, most = 2 * kSMs / blocks > 1 ? 2 * kSMs / blocks : 1;
    return (int)(pieces < most ? pieces : most);
}

cudaError_t launch_conv_bwd(const ConvArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return conv::backward<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return conv::backward<__half>(a, stream);
    return conv::backward<float>(a, stream);
}

}  // namespace kda
