// Layer norm, forward: y = (x - mean) rstd weight + bias over the last dimension, with
// rstd = 1 / sqrt(var + eps), var the mean of the squared differences.
//
// Bound by memory: x is read once and y written once.  The row stays in registers between
// its two passes, so the variance is taken from differences to the mean (no cancellation of
// large sums), in FP32.  Rows of more than 32 threads: each warp finds its own mean and
// squared differences, and one exchange through shared memory joins them,
//   mean = sum n_w mean_w / n,   M2 = sum M2_w + sum n_w (mean_w - mean)^2.
// The next rows are on their way meanwhile (Stream).  32768 x 2048 BF16: 44.4 us, 6.05 TB/s (49.3
// with the sums' operations in pairs, as the backward has them: more registers).
#include "kda_norm.cuh"

namespace kda {
namespace norm {
namespace {

template <typename T, bool WIDE, int TPR>
__global__ void __launch_bounds__(threads<TPR>()) kda_layer_norm_fwd_kernel(const NormArgs a) {
    wait_for_previous();
    constexpr int kThreads = threads<TPR>(), kGroups = kThreads / TPR;
    constexpr int kWarps = TPR > 32 ? TPR / 32 : 1;
    using P = Part<T, WIDE, TPR>;
    constexpr int E = P::E;
    constexpr int R = at_once<WIDE, TPR>(), kDepth = WIDE ? 4 / R + 1 : 2;
    using Rows = Stream<T, WIDE, TPR, kThreads, kDepth * R>;
    __shared__ float2 red[2][kGroups][R][kWarps];
    extern __shared__ __align__(16) char slots[];
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, lane = threadIdx.x & 31;
    const int w = t / 32;
    float wt[E], bs[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = P::col(t, i);
        wt[i] = c < a.width ? param(a.weight, a.wdtype, c, 1.f) : 0.f;
        bs[i] = c < a.width ? param(a.bias, a.wdtype, c, 0.f) : 0.f;
    }
    // elements of the row that warp j of the group holds
    auto held = [&](int j) {
        constexpr int kRun = WIDE ? P::kVec : 1;  // neighbouring columns of a thread
        int n = 0;
#pragma unroll
        for (int i = 0; i < E / kRun; ++i)
            n += min(max(a.width - (i * TPR + j * 32) * kRun, 0), 32 * kRun);
        return n;
    };
    const float inv_n = 1.f / (float)a.width;
    const float inv_w = TPR > 32 ? 1.f / (float)max(held(w), 1) : inv_n;
    const float n_lane = TPR > 32 ? (lane < kWarps ? (float)held(lane) : 0.f) : 0.f;
    const long long step = (long long)gridDim.x * kGroups * R;
    long long row0 = (long long)blockIdx.x * kGroups * R;
    Rows rows(slots);
    auto fetch = [&](int stage, long long first) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long row = first + r * kGroups + grp;
            const bool ok = row < a.rows;
            rows.fetch(stage * R + r, (const T *)a.x + (ok ? row : 0) * a.x_stride, t, a.width, ok,
                       Place(a, row, a.x_stride));
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(i, row0 + i * step);
    for (int it = 0, stage = 0; row0 < a.rows;
         row0 += step, it ^= 1, stage = stage + 1 < kDepth ? stage + 1 : 0) {
        constexpr int kLanes = TPR < 32 ? TPR : 32;
        cp_async_wait_newest<kDepth - 2>();
        float x[R][E], mean[R], m2[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const P cur = rows.take(stage * R + r);
            mean[r] = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) mean[r] += x[r][i] = as_f32(cur.v[i]);
        }
        fetch(stage > 0 ? stage - 1 : kDepth - 1, row0 + (kDepth - 1) * step);
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = lanes_sum<kLanes>(mean[r]) * inv_w;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m2[r] = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float d = x[r][i] - mean[r];
                if (P::col(t, i) < a.width) m2[r] += d * d;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) m2[r] = lanes_sum<kLanes>(m2[r]);
        if (TPR > 32) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (lane == 0) red[it][grp][r][w] = make_float2(mean[r], m2[r]);
            group_sync<TPR>(grp);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 p =
                    lane < kWarps ? red[it][grp][r][lane] : make_float2(0.f, 0.f);
                mean[r] = lanes_sum<32>(p.x * n_lane) * inv_n;
                const float d = p.x - mean[r];
                m2[r] = lanes_sum<32>(p.y + n_lane * d * d);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long row = row0 + r * kGroups + grp;
            const bool ok = row < a.rows;
            const float rstd = rsqrtf(m2[r] * inv_n + a.eps);
            P out;
#pragma unroll
            for (int i = 0; i < E; ++i)
                out.v[i] = from_f32<T>((x[r][i] - mean[r]) * rstd * wt[i] + bs[i]);
            out.store((T *)a.y + row * a.y_stride, t, a.width, ok, Place(a, row, a.y_stride));
            if (ok && t == 0 && dbg_ok(a.dbg, (size_t)row, (size_t)a.rows, DBG_STORE)) {
                if (a.mean) a.mean[row] = mean[r];
                if (a.rstd) a.rstd[row] = rstd;
            }
        }
    }
    cp_async_wait_newest<0>();
}

// Rows that no CTA's registers hold: one CTA a row, three passes over it (from L2).
template <typename T> __global__ void __launch_bounds__(1024) kda_layer_norm_fwd_long_kernel(const NormArgs a) {
    wait_for_previous();
    __shared__ float red[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = (const T *)a.x + row * a.x_stride;
        if (!Place(a, row, a.x_stride).ok(a.width - 1, DBG_LOAD) ||
            !Place(a, row, a.y_stride).ok(a.width - 1, DBG_STORE))
            return;
        float s = 0.f;
        for (int c = tid; c < a.width; c += 1024) s += as_f32(x[c]);
        s = lanes_sum<32>(s);
        if (lane == 0) red[0][warp] = s;
        __syncthreads();
        const float mean = lanes_sum<32>(red[0][lane]) / (float)a.width;
        s = 0.f;
        for (int c = tid; c < a.width; c += 1024) {
            const float d = as_f32(x[c]) - mean;
            s += d * d;
        }
        s = lanes_sum<32>(s);
        if (lane == 0) red[1][warp] = s;
        __syncthreads();
        const float rstd = rsqrtf(lanes_sum<32>(red[1][lane]) / (float)a.width + a.eps);
        T *y = (T *)a.y + row * a.y_stride;
        for (int c = tid; c < a.width; c += 1024)
            y[c] = from_f32<T>((as_f32(x[c]) - mean) * rstd * param(a.weight, a.wdtype, c, 1.f) +
                               param(a.bias, a.wdtype, c, 0.f));
        if (tid == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        __syncthreads();
    }
}

template <typename T, bool WIDE, int TPR>
cudaError_t launch(const NormArgs &a, cudaStream_t stream) {
    constexpr int R = at_once<WIDE, TPR>();
    constexpr int kThreads = threads<TPR>(), kGroups = kThreads / TPR * R;
    constexpr int kBytes = Stream<T, WIDE, TPR, kThreads, (4 / R + 1) * R>::kBytes;
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && kBytes > 40 * 1024)  // with the static part, over the default 48 KB
        e = smem_limit_once(kda_layer_norm_fwd_kernel<T, WIDE, TPR>, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    const long long want = (a.rows + kGroups - 1) / kGroups, most = kSMs * (1024 / kThreads);
    return launch_early(kda_layer_norm_fwd_kernel<T, WIDE, TPR>,
                        (unsigned)(want < most ? want : most), kThreads, kBytes, stream, a);
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
    return launch_early(kda_layer_norm_fwd_long_kernel<T>,
                        (unsigned)(a.rows < most ? a.rows : most), 1024, 0, stream, a);
}

template <typename T> cudaError_t pick_wide(const NormArgs &a, cudaStream_t stream) {
    const bool wide = wide_ok(a.dtype, a.width, a.x, a.x_stride) &&
                      wide_ok(a.dtype, a.width, a.y, a.y_stride);
    return wide ? pick<T, true>(a, stream) : pick<T, false>(a, stream);
}

}  // namespace
}  // namespace norm

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t stream) {
    if (a.dtype == NORM_BF16) return norm::pick_wide<__nv_bfloat16>(a, stream);
    if (a.dtype == NORM_FP16) return norm::pick_wide<__half>(a, stream);
    return norm::pick_wide<float>(a, stream);
}

}  // namespace kda
