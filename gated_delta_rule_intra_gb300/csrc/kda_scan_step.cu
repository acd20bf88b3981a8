// Selective scan, single-token form: one token for each request, its states updated in place
// (kda_scan.cuh has the formulas).
//
// Bound by memory: a state is read once and written once.  A thread has four states of a channel
// and takes that channel of up to four requests, whose states are all asked for before the first is
// used; A is read once for them.
#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

template <typename T, int NP, int R, bool WIDE>
__global__ void __launch_bounds__(kThreads) kda_scan_step_kernel(const ScanArgs a) {
    wait_for_previous();
    using S = Shape<NP>;
    const int c = blockIdx.x * S::HC + threadIdx.x / S::L, part = threadIdx.x % S::L, n0 = 4 * part;
    const int r0 = blockIdx.y * R;
    const bool in = c < a.D;
    const int ch = in ? c : 0, group = ch / (a.D / a.G);
    float *st[R];
    Four h[R];
    bool live[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + i;
        long long slot = r < a.requests ? a.state_indices ? a.state_indices[r] : r : -1;
        live[i] = in && slot >= 0 && slot < a.num_states;
        st[i] = a.state + ((size_t)(live[i] ? slot : 0) * a.D + ch) * a.N;
        h[i] = {both(0.f), both(0.f)};
        if (live[i] && n0 < a.N) {
            if (WIDE)
                h[i] = four(*(const float4 *)(st[i] + n0));
            else
                h[i] = load_states(st[i], 0, n0, a.N, true);
        }
    }
    const Four A2 = scaled(load_states(a.A, ch, n0, a.N, in), kLog2e);
    const float bias = a.delta_bias ? a.delta_bias[ch] : 0.f, skip = a.skip ? a.skip[ch] : 0.f;
    float y[R], u[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        y[i] = u[i] = 0.f;
        if (!live[i]) continue;
        const size_t r = r0 + i;
        u[i] = as_f32(((const T *)a.u)[r * a.u_stride + ch]);
        float d = as_f32(((const T *)a.delta)[r * a.delta_stride + ch]) + bias;
        if (a.softplus) d = softplus(d);
        const T *B = (const T *)a.B + r * a.B_stride + (size_t)group * a.N;
        const T *C = (const T *)a.C + r * a.C_stride + (size_t)group * a.N;
        float b[4], cc[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            b[x] = n0 + x < a.N ? as_f32(B[n0 + x]) : 0.f;
            cc[x] = n0 + x < a.N ? as_f32(C[n0 + x]) : 0.f;
        }
        h[i] = fma(decay(both(d), A2), h[i], mul(both(d * u[i]), four(make_float4(b[0], b[1], b[2], b[3]))));
        y[i] = dot(h[i], four(make_float4(cc[0], cc[1], cc[2], cc[3])));
        if (n0 < a.N) {
            if (WIDE)
                *(float4 *)(st[i] + n0) = one(h[i]);
            else
                store_states(st[i], 0, n0, a.N, h[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int off = S::L / 2; off > 0; off >>= 1) y[i] += __shfl_xor_sync(0xffffffffu, y[i], off);
        const int r = r0 + i;
        if (part == 0 && in && r < a.requests && dbg_ok(a.dbg, (size_t)r, (size_t)a.requests, DBG_STORE)) {
            float out = fmaf(skip, u[i], y[i]);
            if (a.z && live[i]) {
                const float z = as_f32(((const T *)a.z)[(size_t)r * a.z_stride + ch]);
                out *= z * sigmoid(z);
            }
            ((T *)a.y)[(size_t)r * a.y_stride + ch] = from_f32<T>(out);  // a row without a request: zero
        }
    }
}

template <typename T, int NP, int R> cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.D + Shape<NP>::HC - 1) / Shape<NP>::HC), (unsigned)((a.requests + R - 1) / R));
    return a.N % 4 == 0 ? launch_early(kda_scan_step_kernel<T, NP, R, true>, grid, kThreads, 0, stream, a)
                        : launch_early(kda_scan_step_kernel<T, NP, R, false>, grid, kThreads, 0, stream, a);
}
template <typename T, int NP> cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    const long long ctas = (long long)a.requests * ((a.D + Shape<NP>::HC - 1) / Shape<NP>::HC);
    return ctas >= 32 * kSMs ? launch<T, NP, 4>(a, stream) : launch<T, NP, 1>(a, stream);
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
