// Short causal convolution, backward: with g = dy act'(pre), pre computed again from x,
//   dx[t] = sum_j weight[j] g[t + W - 1 - j],
//   dweight[j] = sum over tokens of g[t] x[t - W + 1 + j],  dbias = sum over tokens of g.
// The final state's gradient is that of the sequence's last inputs and is added to theirs.
//
// Bound by memory (x and dy read, dx written once) if instructions leave it room: a resident CTA takes
// pieces of 128 tokens of one block of channels in turn, and the next piece's rows are on their
// way into shared memory meanwhile, whatever their alignment.  A thread walks a run of tokens of four
// channels with the last W inputs and the last W values of g in registers (the places of both go
// round, so that nothing is moved), and W - 1 tokens more whose g its last inputs need.  The CTAs'
// sums of the parameters' gradients are added up in a fixed order by a second kernel.
#include "kda_conv.cuh"

namespace kda {
namespace conv {
namespace {

constexpr int kThreads = 128, V = 4, kPiece = kConvPiece;

template <typename T, int W> struct Smem {
    static constexpr int LANES = 64 / (V * sizeof(T)) * 2;  // of a row: 128 bytes
    static constexpr int CH = LANES * V, kRuns = kThreads / LANES, kRun = kPiece / kRuns;
    static constexpr int kX = kPiece + 2 * (W - 1), kDy = kPiece + W - 1;
    T x[2][kX][CH], dy[2][kDy][CH];
    float w[W + 1][CH], red[kRuns][CH];
};

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 3)
    kda_conv_bwd_kernel(const ConvArgs a, long long pieces, int unit_x, int unit_dy, int unit_dx) {
    wait_for_previous();
    using S = Smem<T, W>;
    extern __shared__ __align__(16) char smem[];
    S &s = *reinterpret_cast<S *>(smem);
    const int tid = threadIdx.x, lane = tid % S::LANES, run = tid / S::LANES;
    const int c0 = blockIdx.x * S::CH, c = c0 + lane * V, left = a.D - c;
    constexpr int kChunks = S::CH / 8;
    // rows of a piece: x from W - 1 in front of it to W - 1 behind, dy from its first token on
    auto fetch = [&](const Piece &p, int b) {
        const int nx = p.len + 2 * (W - 1), ny = p.len + W - 1;
        for (int i = tid; i < nx * kChunks; i += kThreads) {
            const int r = i / kChunks, e = i % kChunks * 8, pos = p.begin - (W - 1) + r;
            const bool front = pos < 0;
            const long long row = front ? (long long)p.seq * (W - 1) + pos + W - 1 : p.row0 + pos;
            const bool ok = pos < p.total && (!front || a.initial) &&
                            dbg_ok(a.dbg, (size_t)row, (size_t)(front ? (long long)a.tok.num_seqs * (W - 1) : a.tok.rows()), DBG_LOAD);
            fetch_chunk<T>((Vec<T, 8> *)&s.x[b][r][e], front && a.initial ? a.initial : a.x,
                           front ? a.D : a.x_stride, ok ? row : 0, c0 + e, a.D - c0 - e, ok, unit_x);
        }
        for (int i = tid; i < ny * kChunks; i += kThreads) {
            const int r = i / kChunks, e = i % kChunks * 8, pos = p.begin + r;
            const long long row = p.row0 + pos;
            const bool ok = pos < p.total && dbg_ok(a.dbg, (size_t)row, (size_t)a.tok.rows(), DBG_LOAD);
            fetch_chunk<T>((Vec<T, 8> *)&s.dy[b][r][e], a.dy, a.dy_stride, ok ? row : 0, c0 + e,
                           a.D - c0 - e, ok, unit_dy);
        }
    };
    for (int i = tid; i < S::CH; i += kThreads) {
        const bool in = c0 + i < a.D;
#pragma unroll
        for (int j = 0; j < W; ++j) s.w[j][i] = in ? param(a.weight, a.wdtype, (size_t)(c0 + i) * W + j, 0.f) : 0.f;
        s.w[W][i] = in ? param(a.bias, a.wdtype, c0 + i, 0.f) : 0.f;
    }
    long long at = blockIdx.y;
    Piece next = at < pieces ? find_piece(a.tok, at, kPiece) : Piece{};
    if (at < pieces && next.len > 0) fetch(next, 0);
    cp_async_commit();
    __syncthreads();
    float w[W][V], bias[V], dw[W][V] = {}, db[V] = {};
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = s.w[j][lane * V + e];
        bias[e] = s.w[W][lane * V + e];
    }
    for (int b = 0; at < pieces; at += gridDim.y, b ^= 1) {
        const Piece p = next;
        if (at + gridDim.y < pieces) {
            next = find_piece(a.tok, at + gridDim.y, kPiece);
            if (next.len > 0) fetch(next, b ^ 1);
        }
        cp_async_commit();
        cp_async_wait_newest<1>();
        __syncthreads();
        const int r0 = run * S::kRun, t0 = p.begin + r0, n = min(S::kRun, p.len - r0);
        if (n > 0 && left > 0) {
            const T *xs = &s.x[b][r0][lane * V], *ys = &s.dy[b][r0][lane * V];
            float xw[W][V], gw[W][V];  // input and g of step i are at i % W
#pragma unroll
            for (int j = 0; j < W - 1; ++j)  // steps -(W - 1) .. -1
                widen(xw[(j + 1) % W], *(const Vec<T, V> *)(xs + j * S::CH));
            T *out = (T *)a.dx + (p.row0 + t0 - (W - 1)) * a.dx_stride + c;
            const int steps = n + W - 1;
            constexpr int U = W == 3 ? 3 : 4;
            for (int base = 0; base < steps; base += U) {
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int i = base + k;  // token t0 + i (i % W = k % W)
                    if (k > 0 && i >= steps) break;
                    float(&x)[V] = xw[k % W], (&g)[V] = gw[k % W];
                    widen(x, *(const Vec<T, V> *)(xs + (i + W - 1) * S::CH));
                    widen(g, *(const Vec<T, V> *)(ys + i * S::CH));
                    if (a.act == ACT_SILU) {
                        float pre[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) pre[e] = bias[e];
#pragma unroll
                        for (int j = 0; j < W; ++j) vfma(pre, xw[(k + 1 + j) % W], w[j]);
                        const bool in = t0 + i < p.total;  // (behind the sequence g is 0)
#pragma unroll
                        for (int e = 0; e < V; e += 2) {
                            const float2 z = make_float2(pre[e], pre[e + 1]);
                            const float2 sg = make_float2(sigmoid(z.x), sigmoid(z.y));
                            const float2 one = make_float2(1.f, 1.f);
                            const float2 sl = mul2(sg, fma2(z, fma2(sg, make_float2(-1.f, -1.f), one), one));
                            const float2 r = mul2(make_float2(g[e], g[e + 1]), sl);
                            g[e] = in ? r.x : 0.f;
                            g[e + 1] = in ? r.y : 0.f;
                        }
                    }
                    if (i < n) {
#pragma unroll
                        for (int j = 0; j < W; ++j) vfma(dw[j], g, xw[(k + 1 + j) % W]);
#pragma unroll
                        for (int e = 0; e < V; e += 2) {
                            const float2 r = add2(make_float2(db[e], db[e + 1]), make_float2(g[e], g[e + 1]));
                            db[e] = r.x;
                            db[e + 1] = r.y;
                        }
                    }
                    if (i >= W - 1) {  // the input W - 1 tokens back has all of its g
                        float dx[V] = {};
#pragma unroll
                        for (int j = 0; j < W; ++j) vfma(dx, w[j], gw[(k + W - j) % W]);
                        const int pos = t0 + i - (W - 1), last = pos - (p.total - (W - 1));
                        if (a.d_final && last >= 0) {
                            const size_t row = (size_t)p.seq * (W - 1) + last;
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                if (e < left && dbg_ok(a.dbg, row, (size_t)a.tok.num_seqs * (W - 1), DBG_LOAD))
                                    dx[e] += as_f32(((const T *)a.d_final)[row * a.D + c + e]);
                        }
                        Vec<T, V> y;
#pragma unroll
                        for (int e = 0; e < V; ++e) y.v[e] = from_f32<T>(dx[e]);
                        if (dbg_ok(a.dbg, (size_t)(p.row0 + pos), (size_t)a.tok.rows(), DBG_STORE)) {
                            T *to = out + i * a.dx_stride;
                            if (unit_dx >= (int)(V * sizeof(T))) {
                                *(Vec<T, V> *)to = y;
                            } else {
#pragma unroll
                                for (int e = 0; e < V; ++e)
                                    if (e < left) to[e] = y.v[e];
                            }
                        }
                    }
                }
            }
        }
        __syncthreads();
    }
    cp_async_wait_newest<0>();
    if (!a.dweight) return;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) s.red[run][lane * V + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
        __syncthreads();
        for (int i = tid; i < S::CH; i += kThreads) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < S::kRuns; ++k) x += s.red[k][i];
            if (c0 + i < a.D && dbg_ok(a.dbg, blockIdx.y, (size_t)a.partials, DBG_STORE))
                a.partial[((size_t)blockIdx.y * (W + 1) + j) * a.D + c0 + i] = x;
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

template <typename T, int W> cudaError_t backward(const ConvArgs &a, cudaStream_t stream) {
    using S = Smem<T, W>;
    const unsigned blocks = (unsigned)((a.D + S::CH - 1) / S::CH);
    const long long pieces = a.tok.pieces(kPiece);
    ConvArgs b = a;  // as many rows of sums as CTAs: one wave, of three a multiprocessor
    const long long most = 3 * kSMs / (long long)blocks > 1 ? 3 * kSMs / (long long)blocks : 1;
    const long long rows = pieces < most ? pieces : most;
    if (rows < b.partials || !a.dweight) b.partials = (int)rows;
    rows::Unit x(sizeof(T), a.D), dy(sizeof(T), a.D), dx(sizeof(T), a.D);
    x.add(a.x, a.x_stride);
    x.add(a.initial, a.D);
    dy.add(a.dy, a.dy_stride);
    dx.add(a.dx, a.dx_stride);
    constexpr int kBytes = sizeof(S);
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = smem_limit_once(kda_conv_bwd_kernel<T, W>, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    e = launch_early(kda_conv_bwd_kernel<T, W>, dim3(blocks, (unsigned)b.partials), kThreads, kBytes, stream, b,
                     pieces, x.unit, dy.unit, dx.unit);
    if (e != cudaSuccess || !a.dweight) return e;
    return launch_early(kda_conv_sum_kernel, (unsigned)(((long long)(W + 1) * a.D + 255) / 256), 256, 0, stream, b);
}
template <typename T> cudaError_t backward(const ConvArgs &a, cudaStream_t stream) {
    if (a.d_initial) {
        const cudaError_t e = launch_early(kda_conv_initial_kernel<T>,
                                           dim3((unsigned)((a.D + 255) / 256), (unsigned)a.tok.num_seqs),
                                           256, 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return a.W == 4 ? backward<T, 4>(a, stream) : a.W == 3 ? backward<T, 3>(a, stream) : backward<T, 2>(a, stream);
}

}  // namespace
}  // namespace conv

// CTAs of a block of channels, each with a row of sums, in the type with the fewest blocks.
int conv_partials(long long pieces, int D) {
    const long long blocks = (D + 63) / 64, most = 3 * kSMs / blocks > 1 ? 3 * kSMs / blocks : 1;
    return (int)(pieces < most ? pieces : most);
}

cudaError_t launch_conv_bwd(const ConvArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return conv::backward<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return conv::backward<__half>(a, stream);
    return conv::backward<float>(a, stream);
}

}  // namespace kda
