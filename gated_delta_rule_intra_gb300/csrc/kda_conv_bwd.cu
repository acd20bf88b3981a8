// Short causal convolution, backward: with g = dy act'(pre), pre computed again from x,
//   dx[t] = sum_j weight[j] g[t + W - 1 - j],
//   dweight[j] = sum over tokens of g[t] x[t - W + 1 + j],  dbias = sum over tokens of g.
// The final state's gradient is that of the sequence's last inputs and is added to theirs.
//
// Bound by instructions (issue slots 56%, four warps a scheduler) next to memory (x and dy read, dx
// written once): 281 us at B=8 T=4096 D=6144 W=4 bf16 with silu, 4.3 TB/s, 63% of a copy's rate.  Rows
// come through shared memory, one piece ahead (kda_conv.cuh).  A thread has the last W values of g in
// registers too, and walks W - 1 tokens more whose g its last inputs need; a whole run is one straight
// piece of code (with a test in every token: 434 us).  Pieces of 96 tokens leave room for four CTAs a
// multiprocessor; pieces of 128, three: 328 us.  Odd rows (9467 tokens of 1111 fp16 channels) take 52 us, 1112
// channels 25: words shifted when read, dx out through shared memory, 36% of the issue slots.  The CTAs'
// sums of the parameters' gradients are added up in a fixed order by a second kernel.
#include <type_traits>

#include "kda_conv.cuh"

namespace kda {
namespace conv {
namespace {

template <typename T, int W, bool ODD> struct Smem {
    using S = Shape<T, ODD>;
    static constexpr int kDy = kPiece + W - 1, kX = kDy + W - 1;
    char x[2][kX][S::kRow], dy[2][kDy][S::kRow];
    float w[W + 1][S::CH], red[S::kRuns][S::CH];
    T dx[kPiece][S::CH];  // only where dx's rows are on no boundary of V elements
};

template <typename T, int W, bool ODD>
__global__ void __launch_bounds__(kThreads, 4)
    kda_conv_bwd_kernel(const ConvArgs a, long long pieces, int unit_x, int unit_dy, int unit_dx) {
    wait_for_previous();
    using S = Shape<T, ODD>;
    using M = Smem<T, W, ODD>;
    extern __shared__ __align__(16) char smem[];
    M &s = *reinterpret_cast<M *>(smem);
    const int tid = threadIdx.x, lane = tid % S::LANES, run = tid / S::LANES;
    const int c0 = blockIdx.x * S::CH, c = c0 + lane * V, left = a.D - c;
    const bool wide = unit_dx >= (int)(V * sizeof(T));
    auto piece = [&](long long at) {
        Piece p;
        p.len = -1;
        return at < pieces ? find_piece(a.tok, at, kPiece) : p;
    };
    // x from W - 1 rows in front of a piece to W - 1 behind it, dy from its first token on
    auto fetch = [&](const Piece &p, int stage) {
        if (p.len > 0) {
            const int end = p.begin + p.len + W - 1;
            fetch_inputs<T, W, ODD>(s.x[stage][0], a, p, end, c0, unit_x);
            fetch_rows<T, ODD>(s.dy[stage][0], a, p, a.dy, a.dy_stride, p.begin, end, c0, unit_dy);
        }
        cp_async_commit();
    };
    load_params<W>(a, c0, s.w);
    Piece next = piece(blockIdx.y);
    fetch(next, 0);
    __syncthreads();
    float w[W][V], bias[V], dw[W][V] = {}, db[V] = {};
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = s.w[j][lane * V + e];
        bias[e] = s.w[W][lane * V + e];
    }
    int b = 0;
    for (long long at = blockIdx.y; at < pieces; at += gridDim.y, b ^= 1) {
        const Piece p = next;
        next = piece(at + gridDim.y);
        fetch(next, b ^ 1);
        cp_async_wait_newest<1>();
        __syncthreads();
        const int r0 = run * S::kRun, t0 = p.begin + r0, n = min(S::kRun, p.len - r0);
        if (n > 0 && left > 0) {
            const char *xs = s.x[b][r0] + lane * V * sizeof(T), *ys = s.dy[b][r0] + lane * V * sizeof(T);
            int xbits[2] = {}, ybits[2] = {};  // of rows an even and an odd number behind the first one
            if (ODD) {
                const long long ex = (p.row0 + t0 - (W - 1)) * a.x_stride + c0, ey = (p.row0 + t0) * a.dy_stride + c0;
                xbits[0] = 16 * shifted<T>(a.x, ex);
                xbits[1] = 16 * shifted<T>(a.x, ex + a.x_stride);
                ybits[0] = 16 * shifted<T>(a.dy, ey);
                ybits[1] = 16 * shifted<T>(a.dy, ey + a.dy_stride);
            }
            const bool fin = a.d_final && t0 + n > p.total - (W - 1);  // of the last inputs
            // whole: every token is in the sequence, the W - 1 behind the run too
            auto walk = [&](auto whole) {
                float xw[W][V], gw[W][V];  // input and g of step i are at i % W
                T *out = wide ? (T *)a.dx + (p.row0 + t0) * a.dx_stride + c : &s.dx[r0][lane * V];
                const long long step = wide ? a.dx_stride : S::CH;
#pragma unroll
                for (int j = 0; j < W - 1; ++j)  // steps -(W - 1) .. -1
                    widen(xw[(j + 1) % W], take<T, ODD>(xs + j * S::kRow, xbits[j & 1]));
#pragma unroll
                for (int i = 0; i < S::kRun + W - 1; ++i) {  // token t0 + i
                    if (!whole && i >= n + W - 1) break;
                    float(&x)[V] = xw[i % W], (&g)[V] = gw[i % W];
                    widen(x, take<T, ODD>(xs + (i + W - 1) * S::kRow, xbits[(i + W - 1) & 1]));
                    widen(g, take<T, ODD>(ys + i * S::kRow, ybits[i & 1]));
                    if (a.act == ACT_SILU) {
                        float pre[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) pre[e] = bias[e];
#pragma unroll
                        for (int j = 0; j < W; ++j) vfma(pre, xw[(i + 1 + j) % W], w[j]);
#pragma unroll
                        for (int e = 0; e < V; e += 2) {
                            const float2 z = make_float2(pre[e], pre[e + 1]);
                            const float2 sg = make_float2(sigmoid(z.x), sigmoid(z.y));
                            const float2 one = make_float2(1.f, 1.f);
                            const float2 sl = mul2(sg, fma2(z, fma2(sg, make_float2(-1.f, -1.f), one), one));
                            const float2 r = mul2(make_float2(g[e], g[e + 1]), sl);
                            g[e] = r.x;
                            g[e + 1] = r.y;
                        }
                        if (!whole && t0 + i >= p.total) {  // behind the sequence, whatever its last inputs are
#pragma unroll
                            for (int e = 0; e < V; ++e) g[e] = 0.f;
                        }
                    }
                    if (whole ? i < S::kRun : i < n) {
#pragma unroll
                        for (int j = 0; j < W; ++j) vfma(dw[j], g, xw[(i + 1 + j) % W]);
#pragma unroll
                        for (int e = 0; e < V; e += 2) {
                            const float2 r = add2(make_float2(db[e], db[e + 1]), make_float2(g[e], g[e + 1]));
                            db[e] = r.x;
                            db[e + 1] = r.y;
                        }
                    }
                    if (i < W - 1) continue;
                    float dx[V] = {};  // of the input W - 1 tokens back, which has all of its g
#pragma unroll
                    for (int j = 0; j < W; ++j) vfma(dx, w[j], gw[(i + W - j) % W]);
                    const int pos = t0 + i - (W - 1), last = pos - (p.total - (W - 1));
                    if (!whole && fin && last >= 0) {
                        const size_t row = (size_t)p.seq * (W - 1) + last;
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (e < left && in_bounds(a.dbg, row, (size_t)a.tok.num_seqs * (W - 1), DBG_LOAD))
                                dx[e] += as_f32(((const T *)a.d_final)[row * a.D + c + e]);
                    }
                    Vec<T, V> y;
                    narrow(y, dx);
                    if (in_bounds(a.dbg, (size_t)(p.row0 + pos), (size_t)a.tok.rows(), DBG_STORE))
                        *(Vec<T, V> *)out = y;
                    out += step;
                }
            };
            if (n == S::kRun && t0 + n + W - 1 <= p.total)
                walk(std::true_type());
            else
                walk(std::false_type());
        }
        __syncthreads();
        if (!wide && p.len > 0) leave_rows<T, S::CH>(s.dx, a, p, a.dx, a.dx_stride, c0);
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
            const size_t at = ((size_t)blockIdx.y * (W + 1) + j) * a.D + c0 + i;
            if (c0 + i < a.D && in_bounds(a.dbg, at, a.partial_floats, DBG_STORE)) a.partial[at] = x;
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
    for (int k = 0; k < a.partials; ++k) {
        const size_t at = ((size_t)k * (a.W + 1) + j) * a.D + c;
        if (in_bounds(a.dbg, at, a.partial_floats, DBG_LOAD)) s += a.partial[at];
    }
    if (j < a.W) {
        if (in_bounds(a.dbg, (size_t)c * a.W + j, (size_t)a.D * a.W, DBG_STORE)) a.dweight[(size_t)c * a.W + j] = s;
    } else if (in_bounds(a.dbg, (size_t)c, (size_t)a.D, DBG_STORE)) {
        a.dbias[c] = s;
    }
}

// Gradients of the inputs in front of each sequence: its first W - 1 values of g again.
template <typename T> __global__ void __launch_bounds__(256) kda_conv_initial_kernel(const ConvArgs a) {
    wait_for_previous();
    const int blocks = (a.D + 255) / 256, c = blockIdx.x % blocks * 256 + threadIdx.x, n = blockIdx.x / blocks, W = a.W;
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
    auto row_ok = [&](int pos) { return in_bounds(a.dbg, (size_t)(p.row0 + pos), (size_t)a.tok.rows(), DBG_LOAD); };
    auto state = [&](const void *of, int row) {
        const size_t at = (size_t)n * (W - 1) + row;
        return in_bounds(a.dbg, at, (size_t)a.tok.num_seqs * (W - 1), DBG_LOAD) ? as_f32(((const T *)of)[at * a.D + c]) : 0.f;
    };
    auto input = [&](int pos) {
        return pos >= 0 ? row_ok(pos) ? as_f32(((const T *)a.x)[(p.row0 + pos) * a.x_stride + c]) : 0.f
               : a.initial ? state(a.initial, pos + W - 1) : 0.f;
    };
    float d[3] = {};
    for (int t = 0; t < W - 1 && t < p.total; ++t) {
        float g = row_ok(t) ? as_f32(((const T *)a.dy)[(p.row0 + t) * a.dy_stride + c]) : 0.f;
        if (a.act == ACT_SILU) {
            float pre = param(a.bias, a.wdtype, c, 0.f);
            for (int j = 0; j < W; ++j)
                pre = fmaf(input(t - (W - 1) + j),
                           param(a.weight, a.wdtype, (size_t)c * W + j, 0.f), pre);
            g *= silu_slope(pre, sigmoid(pre));
        }
        for (int r = t; r < W - 1; ++r)  // input r - (W - 1) is token t's tap r - t
            d[r] = fmaf(g, param(a.weight, a.wdtype, (size_t)c * W + r - t, 0.f), d[r]);
    }
    for (int r = 0; r < W - 1; ++r) {
        const int last = r - p.total;  // where it is still among the last inputs
        if (a.d_final && last >= 0) d[r] += state(a.d_final, last);
        if (in_bounds(a.dbg, (size_t)n, (size_t)a.tok.num_seqs, DBG_STORE))
            ((T *)a.d_initial)[((size_t)n * (W - 1) + r) * a.D + c] = from_f32<T>(d[r]);
    }
}

template <typename T, int W, bool ODD>
cudaError_t backward(const ConvArgs &a, int unit_x, int unit_dy, int unit_dx, cudaStream_t stream) {
    using M = Smem<T, W, ODD>;
    const unsigned blocks = (unsigned)((a.D + M::S::CH - 1) / M::S::CH);
    const long long pieces = a.tok.pieces(kPiece);
    constexpr int kBytes = sizeof(M);
    const int bytes = unit_dx >= (int)(V * sizeof(T)) ? kBytes - (int)sizeof(M::dx) : kBytes;
    ConvArgs b = a;  // as many rows of sums as CTAs: one wave
    const long long wave = resident(bytes, 4) * kSMs / blocks, most = wave > 1 ? wave : 1;
    const long long rows = pieces < most ? pieces : most;
    if (rows < b.partials || !a.dweight) b.partials = (int)rows;
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = smem_limit_once(kda_conv_bwd_kernel<T, W, ODD>, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    e = launch_early(kda_conv_bwd_kernel<T, W, ODD>, dim3(blocks, (unsigned)b.partials), kThreads, bytes, stream, b,
                     pieces, unit_x, unit_dy, unit_dx);
    if (e != cudaSuccess || !a.dweight) return e;
    return launch_early(kda_conv_sum_kernel, (unsigned)(((long long)(W + 1) * a.D + 255) / 256), 256, 0, stream, b);
}
template <typename T, int W> cudaError_t backward(const ConvArgs &a, cudaStream_t stream) {
    rows::Boundary x(sizeof(T), 16), dy(sizeof(T), 16), dx(sizeof(T), a.D);
    x.add(a.x, a.x_stride);
    dy.add(a.dy, a.dy_stride);
    dx.add(a.dx, a.dx_stride);
    if constexpr (sizeof(T) == 2)
        if (x.unit < 4 || dy.unit < 4) return backward<T, W, true>(a, x.unit, dy.unit, dx.unit, stream);
    return backward<T, W, false>(a, x.unit, dy.unit, dx.unit, stream);
}
template <typename T> cudaError_t backward(const ConvArgs &a, cudaStream_t stream) {
    if (a.d_initial) {
        const cudaError_t e = launch_early(kda_conv_initial_kernel<T>,
                                           (unsigned)((a.D + 255) / 256 * (long long)a.tok.num_seqs), 256, 0,
                                           stream, a);
        if (e != cudaSuccess) return e;
    }
    return a.W == 4 ? backward<T, 4>(a, stream) : a.W == 3 ? backward<T, 3>(a, stream) : backward<T, 2>(a, stream);
}

}  // namespace
}  // namespace conv

// CTAs of a block of channels, each with a row of sums, in the type with the fewest blocks.
int conv_partials(long long pieces, int D) {
    const long long blocks = (D + 63) / 64, most = 4 * kSMs / blocks > 1 ? 4 * kSMs / blocks : 1;
    return (int)(pieces < most ? pieces : most);
}

cudaError_t launch_conv_bwd(const ConvArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return conv::backward<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return conv::backward<__half>(a, stream);
    return conv::backward<float>(a, stream);
}

}  // namespace kda
