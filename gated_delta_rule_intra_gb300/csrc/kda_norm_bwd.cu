// Layer norm, backward: with xhat = (x - mean) rstd and h = dy weight,
//   dx = rstd (h - mean(h) - xhat mean(h xhat)),
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy.
//
// Bound by memory: x and dy are read once, dx is written once.  A resident CTA walks rows
// grid-stride and keeps its columns' sums of dy xhat and dy in registers; at the end it writes
// them to its own row of `partial`, and a second kernel adds the rows up in a fixed order, so
// the result does not depend on which CTA finished first.  32768 x 2048 BF16: 68.3 + 3.4 us, of
// which the first is 5.9 TB/s.
#include "kda_norm.cuh"

namespace kda {
namespace norm {
namespace {

// CTAs a multiprocessor, and rows on their way to a thread (the widest FP32 rows: 192 KB of
// slots).  One row at a time: two at once, as in the forward, spill.
template <int E, bool WIDE, int TPR> constexpr int per_sm() {
    return TPR > 256 ? 1 : WIDE && E == 8 ? 3 : 2;
}
template <bool WIDE, int TPR> constexpr int depth() { return !WIDE ? 2 : TPR == 1024 ? 3 : 4; }

template <typename T, bool WIDE, int TPR>
__global__ void __launch_bounds__(threads<TPR>(), per_sm<elements<T, WIDE>(), WIDE, TPR>())
    kda_layer_norm_bwd_kernel(const NormArgs a) {
    wait_for_previous();
    constexpr int kThreads = threads<TPR>(), kGroups = kThreads / TPR;
    constexpr int kWarps = TPR > 32 ? TPR / 32 : 1;
    using P = Part<T, WIDE, TPR>;
    constexpr int E = P::E, kDepth = depth<WIDE, TPR>();
    using Rows = Stream<T, WIDE, TPR, kThreads, kDepth>;
    __shared__ float2 red[2][kGroups][kWarps];
    extern __shared__ __align__(16) char slots[];
    __shared__ float sums[kGroups > 1 ? kGroups : 1][kGroups > 1 ? TPR * E : 1];
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, lane = threadIdx.x & 31;
    const int w = t / 32;
    float2 wt[E / 2], dw[E / 2] = {}, db[E / 2] = {};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = P::col(t, i);
        (i & 1 ? wt[i / 2].y : wt[i / 2].x) =
            c < a.width ? param(a.weight, a.wdtype, c, 1.f) : 0.f;
    }
    const float inv_n = 1.f / (float)a.width;
    const long long step = (long long)gridDim.x * kGroups;
    long long row0 = (long long)blockIdx.x * kGroups;
    Rows xs(slots), dys(slots + Rows::kBytes);
    auto fetch = [&](int stage, long long row) {
        const bool ok = row < a.rows;
        const long long at = ok ? row : 0;
        xs.fetch(stage, (const T *)a.x + at * a.x_stride, t, a.width, ok, Place(a, row, a.x_stride));
        dys.fetch(stage, (const T *)a.dy + at * a.dy_stride, t, a.width, ok,
                  Place(a, row, a.dy_stride));
        cp_async_commit();
    };
    auto stats = [&](long long row) {
        return row < a.rows && dbg_ok(a.dbg, (size_t)row, (size_t)a.rows, DBG_LOAD)
                   ? make_float2(a.mean[row], a.rstd[row]) : make_float2(0.f, 0.f);
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(i, row0 + i * step + grp);
    float2 st = stats(row0 + grp), st1 = stats(row0 + step + grp);
    for (int it = 0, stage = 0; row0 < a.rows;
         row0 += step, it ^= 1, stage = stage + 1 < kDepth ? stage + 1 : 0) {
        const long long row = row0 + grp;
        cp_async_wait_newest<kDepth - 2>();
        const P x = xs.take(stage), dy = dys.take(stage);
        fetch(stage > 0 ? stage - 1 : kDepth - 1, row + (kDepth - 1) * step);
        const float mean = st.x, rstd = st.y;
        st = st1;
        st1 = stats(row + 2 * step);
        // past the row's end weight and dy are zero, so that nothing of xhat there counts
        float2 sum1 = both(0.f), sum2 = both(0.f), xh[E / 2], h[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 d = two(&dy.v[2 * i]);
            xh[i] = mul2(add2(two(&x.v[2 * i]), both(-mean)), both(rstd));
            h[i] = mul2(d, wt[i]);
            sum1 = add2(sum1, h[i]);
            sum2 = fma2(h[i], xh[i], sum2);
            dw[i] = fma2(d, xh[i], dw[i]);
            db[i] = add2(db[i], d);
        }
        float s1 = sum1.x + sum1.y, s2 = sum2.x + sum2.y;
        constexpr int kLanes = TPR < 32 ? TPR : 32;
        s1 = lanes_sum<kLanes>(s1);
        s2 = lanes_sum<kLanes>(s2);
        if (TPR > 32) {
            if (lane == 0) red[it][grp][w] = make_float2(s1, s2);
            group_sync<TPR>(grp);
            const float2 p = lane < kWarps ? red[it][grp][lane] : make_float2(0.f, 0.f);
            s1 = lanes_sum<32>(p.x);
            s2 = lanes_sum<32>(p.y);
        }
        s1 *= inv_n;
        s2 *= inv_n;
        P out;
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            put_two(&out.v[2 * i], mul2(both(rstd), fma2(xh[i], both(-s2), add2(h[i], both(-s1)))));
        out.store((T *)a.dx + row * a.dx_stride, t, a.width, row < a.rows,
                  Place(a, row, a.dx_stride));
    }
    cp_async_wait_newest<0>();
    if (!a.dweight || !dbg_ok(a.dbg, blockIdx.x, (size_t)a.partials, DBG_STORE)) return;
    float *to = a.partial + (size_t)blockIdx.x * 2 * a.width;
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = P::col(t, i);
            if (c < a.width) {
                to[c] = i & 1 ? dw[i / 2].y : dw[i / 2].x;
                to[a.width + c] = i & 1 ? db[i / 2].y : db[i / 2].x;
            }
        }
    } else {
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float2 x = pass ? db[i / 2] : dw[i / 2];
                sums[grp][P::col(t, i)] = i & 1 ? x.y : x.x;
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.width; c += kThreads) {
                float s = 0.f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) s += sums[g][c];
                to[pass * a.width + c] = s;
            }
        }
    }
}

// Column sums of `partial` [n][cols]: 32 columns a CTA, 32 slices of rows side by side.
__global__ void __launch_bounds__(1024)
    kda_layer_norm_sum_kernel(const float *partial, int n, int width, float *dweight, float *dbias,
                              int partials, unsigned *dbg) {
    wait_for_previous();
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const long long cols = 2LL * width, c = (long long)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols && dbg_ok(dbg, (size_t)n, (size_t)partials + 1, DBG_LOAD)) {
#pragma unroll 4
        for (int i = slice; i < n; i += 32) s += partial[(size_t)i * cols + c];
    }
    red[slice][lane] = s;
    __syncthreads();
    s = lanes_sum<32>(red[lane][slice]);
    const long long col = (long long)blockIdx.x * 32 + slice;
    if (lane == 0 && col < cols) {
        if (col < width)
            dweight[col] = s;
        else
            dbias[col - width] = s;
    }
}

// Rows that no CTA's registers hold: dx by one CTA a row ...
template <typename T> __global__ void __launch_bounds__(1024) kda_layer_norm_bwd_long_kernel(const NormArgs a) {
    wait_for_previous();
    __shared__ float2 red[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = (const T *)a.x + row * a.x_stride, *dy = (const T *)a.dy + row * a.dy_stride;
        if (!Place(a, row, a.x_stride).ok(a.width - 1, DBG_LOAD) ||
            !Place(a, row, a.dy_stride).ok(a.width - 1, DBG_LOAD) ||
            !Place(a, row, a.dx_stride).ok(a.width - 1, DBG_STORE))
            return;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.f, s2 = 0.f;
        for (int c = tid; c < a.width; c += 1024) {
            const float h = as_f32(dy[c]) * param(a.weight, a.wdtype, c, 1.f);
            s1 += h;
            s2 += h * (as_f32(x[c]) - mean) * rstd;
        }
        s1 = lanes_sum<32>(s1);
        s2 = lanes_sum<32>(s2);
        if (lane == 0) red[warp] = make_float2(s1, s2);
        __syncthreads();
        s1 = lanes_sum<32>(red[lane].x) / (float)a.width;
        s2 = lanes_sum<32>(red[lane].y) / (float)a.width;
        T *dx = (T *)a.dx + row * a.dx_stride;
        for (int c = tid; c < a.width; c += 1024) {
            const float xh = (as_f32(x[c]) - mean) * rstd;
            dx[c] = from_f32<T>(
                rstd * (as_f32(dy[c]) * param(a.weight, a.wdtype, c, 1.f) - s1 - xh * s2));
        }
        __syncthreads();
    }
}

// ... and the column sums by a pass of their own: 256 columns a CTA, one slice of the rows.
template <typename T> __global__ void __launch_bounds__(256) kda_layer_norm_bwd_cols_kernel(const NormArgs a) {
    wait_for_previous();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.width || !dbg_ok(a.dbg, blockIdx.y, (size_t)a.partials, DBG_STORE)) return;
    float dw = 0.f, db = 0.f;
    for (long long row = blockIdx.y; row < a.rows; row += gridDim.y) {
        if (!Place(a, row, a.dy_stride).ok(c, DBG_LOAD) || !Place(a, row, a.x_stride).ok(c, DBG_LOAD))
            return;
        const float d = as_f32(((const T *)a.dy)[row * a.dy_stride + c]);
        dw += d * (as_f32(((const T *)a.x)[row * a.x_stride + c]) - a.mean[row]) * a.rstd[row];
        db += d;
    }
    float *to = a.partial + (size_t)blockIdx.y * 2 * a.width;
    to[c] = dw;
    to[a.width + c] = db;
}

// CTAs, each with a row of `partial`.
int ctas(long long rows, int width, int e, bool wide) {
    const int tpr = group_of(width, e);
    if (!tpr) return (int)(rows < 64 ? rows : 64);  // slices of the column pass
    const int groups = tpr < 256 ? 256 / tpr : 1;
    const int a_sm = tpr > 256 ? 1024 / tpr : wide && e == 8 ? 3 : 2;
    const long long want = (rows + groups - 1) / groups, most = (long long)kSMs * a_sm;
    return (int)(want < most ? want : most);
}

cudaError_t sum_partials(const NormArgs &a, int n, cudaStream_t stream) {
    if (!a.dweight) return cudaSuccess;
    return launch_early(kda_layer_norm_sum_kernel, (unsigned)((2LL * a.width + 31) / 32), 1024, 0,
                        stream, a.partial, n, a.width, a.dweight, a.dbias, a.partials, a.dbg);
}

template <typename T, bool WIDE, int TPR>
cudaError_t launch(const NormArgs &a, cudaStream_t stream) {
    constexpr int kBytes = 2 * Stream<T, WIDE, TPR, threads<TPR>(), depth<WIDE, TPR>()>::kBytes;
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && kBytes > 40 * 1024)  // with the static part, over the default 48 KB
        e = smem_limit_once(kda_layer_norm_bwd_kernel<T, WIDE, TPR>, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    const int n = ctas(a.rows, a.width, elements<T, WIDE>(), WIDE);
    e = launch_early(kda_layer_norm_bwd_kernel<T, WIDE, TPR>, n, threads<TPR>(), kBytes, stream, a);
    return e != cudaSuccess ? e : sum_partials(a, n, stream);
}

template <typename T, bool WIDE> cudaError_t pick(const NormArgs &a, cudaStream_t stream) {
    constexpr int E = elements<T, WIDE>();
    switch (group_of(a.width, E)) {
        case 128 / E: return launch<T, WIDE, 128 / E>(a, stream);
        case 256 / E: return launch<T, WIDE, 256 / E>(a, stream);
        case 512 / E: return launch<T, WIDE, 512 / E>(a, stream);
        case 1024 / E: return launch<T, WIDE, 1024 / E>(a, stream);
        case 2048 / E: return launch<T, WIDE, 2048 / E>(a, stream);
        case 4096 / E: return launch<T, WIDE, 4096 / E>(a, stream);
        case 8192 / E: return launch<T, WIDE, 8192 / E>(a, stream);
    }
    const long long most = 2 * kSMs;
    cudaError_t e = launch_early(kda_layer_norm_bwd_long_kernel<T>,
                                 (unsigned)(a.rows < most ? a.rows : most), 1024, 0, stream, a);
    if (e != cudaSuccess || !a.dweight) return e;
    const int n = ctas(a.rows, a.width, elements<T, WIDE>(), WIDE);
    e = launch_early(kda_layer_norm_bwd_cols_kernel<T>,
                     dim3((unsigned)((a.width + 255) / 256), (unsigned)n), 256, 0, stream, a);
    return e != cudaSuccess ? e : sum_partials(a, n, stream);
}

template <typename T> cudaError_t pick_wide(const NormArgs &a, cudaStream_t stream) {
    const bool wide = wide_ok(a.dtype, a.width, a.x, a.x_stride) &&
                      wide_ok(a.dtype, a.width, a.dy, a.dy_stride) &&
                      wide_ok(a.dtype, a.width, a.dx, a.dx_stride);
    return wide ? pick<T, true>(a, stream) : pick<T, false>(a, stream);
}

}  // namespace
}  // namespace norm

// Enough for rows of any type and alignment.
int norm_bwd_ctas(long long rows, int width) {
    int most = 0;
    for (int e = 8; e <= 16; e *= 2)
        for (int wide = 0; wide < 2; ++wide) {
            const int n = norm::ctas(rows, width, e, wide);
            most = n > most ? n : most;
        }
    return most;
}

cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t stream) {
    if (a.rows == 0) return norm::sum_partials(a, 0, stream);  // sums of nothing: zeros
    if (a.dtype == NORM_BF16) return norm::pick_wide<__nv_bfloat16>(a, stream);
    if (a.dtype == NORM_FP16) return norm::pick_wide<__half>(a, stream);
    return norm::pick_wide<float>(a, stream);
}

}  // namespace kda
