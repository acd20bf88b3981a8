// Selective scan, single-token form: one token for each request, its states updated in place
// (kda_scan.cuh has the formulas).
//
// Bound by memory: a state is read once and written once.  A thread has four states of a channel.
// Where there are requests enough it takes that channel of four of them: their states are all asked for
// before the first is used, A is read once for them, and the lanes of a channel share out what
// there is once a request and channel (the step size, the input, the gate, the result).  The states are
// marked as not to be kept in L2: they come again when all other layers' have been through it.  256
// requests of 4096 channels, 16 states each (142 MB in all): 33 us with states from memory, 45 without
// the mark, 4.3 TB/s (a copy of that much takes 25); one request a thread takes 37.
#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

// Four numbers of B or C from n0 on; zeros from N on.
template <typename T, bool WIDE>
__device__ __forceinline__ Four vector_of(const void *base, long long at, int n0, int N) {
    const T *v = (const T *)base + at + n0;
    if (WIDE) {
        const Vec<T, 4> x = *(const Vec<T, 4> *)v;
        return {x.two(0), x.two(2)};
    }
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = n0 + i < N ? as_f32(v[i]) : 0.f;
    return four(make_float4(f[0], f[1], f[2], f[3]));
}

// WIDE: N is a multiple of 4, and so is where rows of B and C begin.
template <typename T, int NP, int R, bool WIDE>
__global__ void __launch_bounds__(kThreads, R == 4 ? 6 : 1) kda_scan_step_kernel(const ScanArgs a) {
    wait_for_previous();
    using S = Shape<NP>;
    // the requests of this lane: all of them, or its share
    constexpr int kMine = R == 4 ? Share<S::L>::kCount : R;
    const int c = blockIdx.x * S::HC + threadIdx.x / S::L, part = threadIdx.x % S::L, n0 = 4 * part;
    const int r0 = blockIdx.y * R, mine = R == 4 ? Share<S::L>::first(part) : 0;
    const bool in = c < a.D, some = n0 < a.N;
    const int ch = in ? c : 0;
    const long long group = (long long)(ch / (a.D / a.G)) * a.N;
    float *st[R];
    Four h[R], B[R], C[R];
    unsigned live = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + i;
        const long long slot = r < a.requests ? a.state_indices ? a.state_indices[r] : r : -1;
        if (slot >= 0 && slot < a.num_states &&
            in_bounds(a.dbg, ((size_t)slot * a.D + ch) * a.N + a.N - 1, (size_t)a.num_states * a.D * a.N, DBG_STORE))
            live |= 1u << i;
        st[i] = a.state + ((size_t)(live >> i & 1 ? slot : 0) * a.D + ch) * a.N + n0;
        h[i] = {both(0.f), both(0.f)};
        if ((live >> i & 1) && in && some) h[i] = WIDE ? four(__ldcs((const float4 *)st[i])) : load_states(st[i], 0, 0, a.N - n0, true);
    }
    float u[kMine], d[kMine], z[kMine];
    const float bias = a.delta_bias ? a.delta_bias[ch] : 0.f, skip = a.skip ? a.skip[ch] : 0.f;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const long long r = min(r0 + mine + i, a.requests - 1);
        u[i] = as_f32(((const T *)a.u)[r * a.u_stride + ch]);
        d[i] = as_f32(((const T *)a.delta)[r * a.delta_stride + ch]) + bias;
        z[i] = a.z ? as_f32(((const T *)a.z)[r * a.z_stride + ch]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const long long r = min(r0 + i, a.requests - 1);
        B[i] = C[i] = {both(0.f), both(0.f)};
        if (some) {
            B[i] = vector_of<T, WIDE>(a.B, r * a.B_stride + group, n0, a.N);
            C[i] = vector_of<T, WIDE>(a.C, r * a.C_stride + group, n0, a.N);
        }
    }
    const Four A2 = scaled(load_states(a.A, ch, n0, a.N, in), kLog2e);
    const float slowest = slowest_of(A2, n0, a.N, 0);
    if (a.softplus) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) d[i] = softplus(d[i]);
    }
    float y[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float di = d[i % kMine], ui = u[i % kMine];
        if (R == 4 && S::L > 1) {  // from the lane that has this request
            constexpr int kEach = S::L > 4 ? S::L / 4 : 1;  // lanes of one request
            const int from = i / kMine * kEach;
            di = __shfl_sync(0xffffffffu, di, from, S::L);
            ui = __shfl_sync(0xffffffffu, ui, from, S::L);
        }
        h[i] = fma(decay(both(di), A2, raise_of(fabsf(di) * slowest)), h[i], mul(both(di * ui), B[i]));
        y[i] = dot(h[i], C[i]);
        if ((live >> i & 1) && in && some) {
            if (WIDE)
                __stcs((float4 *)st[i], one(h[i]));
            else
                store_states(st[i], 0, 0, a.N - n0, h[i]);
        }
    }
    if (R == 4) {
        scatter_sum<S::L, 1>(y, threadIdx.x);
    } else {
#pragma unroll
        for (int off = S::L / 2; off > 0; off >>= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], off);
    }
    if (!in || !(R == 4 ? Share<S::L>::mine(part) : part == 0)) return;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = r0 + mine + i;
        if (r >= a.requests || !in_bounds(a.dbg, (size_t)r, (size_t)a.requests, DBG_STORE)) continue;
        float out = fmaf(skip, u[i], y[i]);
        if (a.z) out *= z[i] * sigmoid(z[i]);
        if (!(live >> (mine + i) & 1)) out = 0.f;  // a row without a request
        ((T *)a.y)[(size_t)r * a.y_stride + ch] = from_f32<T>(out);
    }
}

template <typename T, int NP, int R> cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.D + Shape<NP>::HC - 1) / Shape<NP>::HC), (unsigned)((a.requests + R - 1) / R));
    const size_t four = 4 * (size_t)esize(a.dtype);
    const bool wide = a.N % 4 == 0 && aligned(a.B, four) && aligned(a.C, four) && a.B_stride % 4 == 0 && a.C_stride % 4 == 0;
    return wide ? launch_early(kda_scan_step_kernel<T, NP, R, true>, grid, kThreads, 0, stream, a)
                        : launch_early(kda_scan_step_kernel<T, NP, R, false>, grid, kThreads, 0, stream, a);
}
template <typename T, int NP> cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    const long long ctas = (long long)a.requests * ((a.D + Shape<NP>::HC - 1) / Shape<NP>::HC);
    // 4096 channels, four requests a thread and one: 16 requests 3.8 and 3.9 us, 32 5.8 and 6.2, 8 3.1 and
    // 3.1, 4 2.8 and 2.3
    return ctas >= 16 * kSMs ? launch<T, NP, 4>(a, stream) : launch<T, NP, 1>(a, stream);
}

template <typename T> cudaError_t pick(const ScanArgs &a, cudaStream_t stream) {
    switch (scan_padded(a.N)) {
        case 8: return launch<T, 8>(a, stream);
        case 16: return launch<T, 16>(a, stream);
        case 32: return launch<T, 32>(a, stream);
    }
    return launch<T, 64>(a, stream);
}

}  // namespace
}  // namespace scan

cudaError_t launch_scan_step(const ScanArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return scan::pick<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return scan::pick<__half>(a, stream);
    return scan::pick<float>(a, stream);
}

}  // namespace kda
