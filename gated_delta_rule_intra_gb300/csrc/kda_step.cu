// The recurrence's single-token form: one token for each request, its state updated in place.
//
//   S~ = diag(2^gate) S,  u = S~^T k,  n = beta (v - u),  S' = S~ + k n^T,
//   o = scale S'^T q = scale (S~^T q + (q . k) n)
//
// The state (64 KB a head in FP32) is read once and written once; everything else is 1.5 KB.
// A CTA holds its part of one head's state in registers between the column sums and the
// update, every load issued before the first use.  Bound by memory: 8192 heads take 156 us,
// 6.9 TB/s; one request's 16 heads take 2.5 us, the latency of a launch and one round trip.
#include "kda_chunk.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int D = KD;

// VQ: groups of four dv columns of a CTA (32 = the whole head).
template <typename T16, int VQ>
__global__ void __launch_bounds__(kThreads) kda_step_kernel(const StepArgs a) {
    wait_for_previous();
    constexpr int kRowGroups = kThreads / VQ;  // dk rows in flight side by side
    constexpr int kRows = D / kRowGroups;      // rows of a thread
    __shared__ float coef[3][D];               // 2^gate, k, q
    __shared__ float qk_part[4];
    __shared__ float4 part[kThreads / 32][2][VQ];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / (32 / VQ), c0 = (blockIdx.x % (32 / VQ)) * VQ;
    const int n = unit / a.HV, hv = unit - n * a.HV, h = hv / (a.HV / a.H);
    const int quad = tid % VQ, rg = tid / VQ;
    const size_t row = (size_t)n * a.HV + hv;
    long long slot = n;
    if (a.state_indices) {
        slot = a.state_indices[n];
        if (slot < 0 || slot >= a.num_states) {  // no request here: o is zero
            const size_t idx = row * D + 4 * (c0 + quad);
            if (rg == 0 && dbg_ok(a.dbg, idx + 3, (size_t)a.N * a.HV * D, DBG_STORE))
                *reinterpret_cast<uint2 *>((uint16_t *)a.o + idx) = make_uint2(0u, 0u);
            return;
        }
    }
    if (!dbg_ok(a.dbg, (size_t)slot * a.HV + hv, (size_t)a.num_states * a.HV, DBG_STORE) ||
        !dbg_ok(a.dbg, row, (size_t)a.N * a.HV, DBG_LOAD))
        return;
    float4 *st = reinterpret_cast<float4 *>(a.state) + ((size_t)slot * a.HV + hv) * (D * D / 4) +
                 c0 + quad;
    float4 s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = st[(size_t)(rg + i * kRowGroups) * (D / 4)];
    const size_t iq = ((size_t)n * a.H + h) * D;
    float qk = 0.f;
    if (tid < D) {
        const float q = to_f32(((const T16 *)a.q)[iq + tid]);
        const float k = to_f32(((const T16 *)a.k)[iq + tid]);
        coef[0][tid] = ex2(chunk::floor_gate(a.gate[row * D + tid]));
        coef[1][tid] = k;
        coef[2][tid] = q;
        qk = q * k;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, off);
        if (lane == 0) qk_part[warp] = qk;
    }
    const float beta = a.beta[row];
    const uint2 vraw = *reinterpret_cast<const uint2 *>((const uint16_t *)a.v + row * D +
                                                        4 * (c0 + quad));
    __syncthreads();
    qk = (qk_part[0] + qk_part[1]) + (qk_part[2] + qk_part[3]);
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = rg + i * kRowGroups;
        const float dec = coef[0][r], k = coef[1][r], q = coef[2][r];
        s[i].x *= dec; s[i].y *= dec; s[i].z *= dec; s[i].w *= dec;
        u.x += k * s[i].x; u.y += k * s[i].y; u.z += k * s[i].z; u.w += k * s[i].w;
        w.x += q * s[i].x; w.y += q * s[i].y; w.z += q * s[i].z; w.w += q * s[i].w;
    }
#pragma unroll
    for (int off = 16; off >= VQ; off >>= 1) {  // row groups inside a warp
        u.x += __shfl_xor_sync(0xffffffffu, u.x, off);
        u.y += __shfl_xor_sync(0xffffffffu, u.y, off);
        u.z += __shfl_xor_sync(0xffffffffu, u.z, off);
        u.w += __shfl_xor_sync(0xffffffffu, u.w, off);
        w.x += __shfl_xor_sync(0xffffffffu, w.x, off);
        w.y += __shfl_xor_sync(0xffffffffu, w.y, off);
        w.z += __shfl_xor_sync(0xffffffffu, w.z, off);
        w.w += __shfl_xor_sync(0xffffffffu, w.w, off);
    }
    if (lane < VQ) {
        part[warp][0][lane] = u;
        part[warp][1][lane] = w;
    }
    __syncthreads();
    u = make_float4(0.f, 0.f, 0.f, 0.f);
    w = u;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        const float4 x = part[i][0][quad], y = part[i][1][quad];
        u.x += x.x; u.y += x.y; u.z += x.z; u.w += x.w;
        w.x += y.x; w.y += y.y; w.z += y.z; w.w += y.w;
    }
    const float2 v0 = chunk::unpack2<T16>(vraw.x), v1 = chunk::unpack2<T16>(vraw.y);
    const float4 e = make_float4(beta * (v0.x - u.x), beta * (v0.y - u.y), beta * (v1.x - u.z),
                                 beta * (v1.y - u.w));
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = rg + i * kRowGroups;
        const float k = coef[1][r];
        s[i].x += k * e.x; s[i].y += k * e.y; s[i].z += k * e.z; s[i].w += k * e.w;
        st[(size_t)r * (D / 4)] = s[i];
    }
    if (rg == 0) {
        uint2 o;
        o.x = chunk::pack2<T16>(a.scale * (w.x + qk * e.x), a.scale * (w.y + qk * e.y));
        o.y = chunk::pack2<T16>(a.scale * (w.z + qk * e.z), a.scale * (w.w + qk * e.w));
        const size_t idx = row * D + 4 * (c0 + quad);
        if (dbg_ok(a.dbg, idx + 3, (size_t)a.N * a.HV * D, DBG_STORE))
            *reinterpret_cast<uint2 *>((uint16_t *)a.o + idx) = o;
    }
}

template <typename T16> cudaError_t launch(const StepArgs &a, cudaStream_t stream) {
    // One CTA a head, or four where that leaves half the SMs without one: 144 heads take 3.9 us in
    // one CTA each and 4.4 in four, 64 heads 3.6 and 3.1.
    const long long heads = (long long)a.N * a.HV;
    if (heads * 2 > kSMs)
        return launch_early(kda_step_kernel<T16, 32>, (unsigned)heads, kThreads, 0, stream, a);
    return launch_early(kda_step_kernel<T16, 8>, (unsigned)(4 * heads), kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_step(const StepArgs &a, cudaStream_t stream) {
    return a.fp16 ? launch<__half>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace kda
