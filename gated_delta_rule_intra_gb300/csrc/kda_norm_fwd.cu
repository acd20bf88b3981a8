// Layer norm, forward: y = (x - mean) rstd weight + bias over the last dimension, with
// rstd = 1 / sqrt(var + eps), var the mean of the squared differences.
//
// Bound by memory: x is read once and y written once.  The row stays in registers between
// its two passes, so the variance is taken from differences to the mean (no cancellation of
// large sums), in FP32.  Rows of more than 32 threads: each warp finds its own mean and
// squared differences, and one exchange through shared memory joins them,
//   mean = sum n_w mean_w / n,   M2 = sum M2_w + sum n_w (mean_w - mean)^2.
// The next row is fetched before the current one's reduction.
#include "kda_norm.cuh"

namespace kda {
namespace norm {
namespace {

template <typename T, bool WIDE, int TPR>
__global__ void __launch_bounds__(threads<TPR>()) kda_layer_norm_fwd_kernel(const NormArgs a) {
    constexpr int kThreads = threads<TPR>(), kGroups = kThreads / TPR;
    constexpr int kWarps = TPR > 32 ? TPR / 32 : 1;
    using P = Part<T, WIDE, TPR>;
    __shared__ float2 red[2][kGroups][kWarps];
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
        if (WIDE) return min(max(a.width - j * 32 * E, 0), 32 * E);
        int n = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) n += min(max(a.width - i * TPR - j * 32, 0), 32);
        return n;
    };
    const float inv_n = 1.f / (float)a.width;
    const float inv_w = TPR > 32 ? 1.f / (float)max(held(w), 1) : inv_n;
    const float n_lane = TPR > 32 ? (lane < kWarps ? (float)held(lane) : 0.f) : 0.f;
    const long long step = (long long)gridDim.x * kGroups;
    long long row0 = (long long)blockIdx.x * kGroups;
    P cur, next;
    cur.load((const T *)a.x + (row0 + grp) * a.x_stride, t, a.width, row0 + grp < a.rows);
    for (int it = 0; row0 < a.rows; row0 += step, it ^= 1) {
        const long long row = row0 + grp;
        const bool ok = row < a.rows, more = row + step < a.rows;
        next.load((const T *)a.x + (row + step) * a.x_stride, t, a.width, more);
        float x[E], s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s += x[i] = as_f32(cur.v[i]);
        constexpr int kLanes = TPR < 32 ? TPR : 32;
        float mean = lanes_sum<kLanes>(s) * inv_w, m2 = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float d = x[i] - mean;
            if (P::col(t, i) < a.width) m2 += d * d;
        }
        m2 = lanes_sum<kLanes>(m2);
        if (TPR > 32) {
            if (lane == 0) red[it][grp][w] = make_float2(mean, m2);
            group_sync<TPR>(grp);
            const float2 p = lane < kWarps ? red[it][grp][lane] : make_float2(0.f, 0.f);
            mean = lanes_sum<32>(p.x * n_lane) * inv_n;
            const float d = p.x - mean;
            m2 = lanes_sum<32>(p.y + n_lane * d * d);
        }
        const float rstd = rsqrtf(m2 * inv_n + a.eps);
        P out;
#pragma unroll
        for (int i = 0; i < E; ++i) out.v[i] = from_f32<T>((x[i] - mean) * rstd * wt[i] + bs[i]);
        out.store((T *)a.y + row * a.y_stride, t, a.width, ok);
        if (ok && t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        cur = next;
    }
}

// Rows that no CTA's registers hold: one CTA a row, three passes over it (from L2).
template <typename T> __global__ void __launch_bounds__(1024) kda_layer_norm_fwd_long_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = (const T *)a.x + row * a.x_stride;
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
    constexpr int kThreads = threads<TPR>(), kGroups = kThreads / TPR;
    const long long want = (a.rows + kGroups - 1) / kGroups, most = kSMs * (2048 / kThreads);
    kda_layer_norm_fwd_kernel<T, WIDE, TPR>
        <<<(unsigned)(want < most ? want : most), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, bool WIDE> cudaError_t pick(const NormArgs &a, cudaStream_t stream) {
    switch (group_of(a.width)) {
        case 16: return launch<T, WIDE, 16>(a, stream);
        case 32: return launch<T, WIDE, 32>(a, stream);
        case 64: return launch<T, WIDE, 64>(a, stream);
        case 128: return launch<T, WIDE, 128>(a, stream);
        case 256: return launch<T, WIDE, 256>(a, stream);
        case 512: return launch<T, WIDE, 512>(a, stream);
        case 1024: return launch<T, WIDE, 1024>(a, stream);
    }
    const long long most = 2 * kSMs;
    kda_layer_norm_fwd_long_kernel<T>
        <<<(unsigned)(a.rows < most ? a.rows : most), 1024, 0, stream>>>(a);
    return cudaGetLastError();
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
