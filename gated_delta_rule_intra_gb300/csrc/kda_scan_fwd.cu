// Selective scan, forward (kda_scan.cuh).
#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

// ENDS: the first pass, which leaves the segments' ends.
template <typename T, int NP, bool ENDS>
__global__ void __launch_bounds__(kThreads) kda_scan_fwd_kernel(const ScanArgs a, int nb, bool vec) {
    wait_for_previous();
    using S = Shape<NP>;
    __shared__ float4 sdx[kTile][S::CH];  // step size twice, step size times input twice
    __shared__ __align__(16) float sB[kTile][NP], sC[kTile][NP], sy[kTile][S::kRow];
    const int tid = threadIdx.x, c = tid / S::L, part = tid % S::L, n0 = 4 * part;
    const Block<NP> k(a, nb);
    const Piece &p = k.p;
    if (p.len < 0 || (ENDS && p.begin + p.len == p.total)) return;
    const bool in = c < k.channels;
    const size_t ch = (size_t)k.c0 + c;
    const Four A2 = scaled(load_states(a.A, ch, n0, a.N, in), kLog2e);
    Four h = {both(0.f), both(0.f)};
    if (!ENDS) {
        h = load_states(a.initial, (size_t)p.seq * a.D + ch, n0, a.N, in && a.initial);
        if (in) {
            for (int j = k.slot - p.index; j < k.slot; ++j) {
                const size_t at = (size_t)j * a.D + ch;
                if (!dbg_ok(a.dbg, at * NP + NP - 1, a.segment_floats, DBG_LOAD)) break;
                h = fma(decay(both(a.sums[at]), A2), h, four(*(const float4 *)(a.ends + at * NP + n0)));
            }
        }
    }
    // this thread's quads of a tile: token q0 + i kThreads / kQuads, channels 4 q ..
    const int q = tid % S::kQuads, qt = tid / S::kQuads, qc = k.c0 + 4 * q, left = k.channels - 4 * q;
    constexpr int kStep = kThreads / S::kQuads;
    float bias[4], skip[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = a.delta_bias && i < left ? a.delta_bias[qc + i] : 0.f;
        skip[i] = a.skip && i < left ? a.skip[qc + i] : 0.f;
    }
    Vec<T, 4> u[S::kPer], dl[S::kPer], z[S::kPer];
    Vectors<T, NP> vb, vc;
    auto fetch = [&](int t0) {
        const int rows = p.len - t0;
        const long long row0 = p.row0 + p.begin + t0;
        const bool fine = rows <= 0 || dbg_ok(a.dbg, (size_t)(row0 + min(rows, kTile) - 1), (size_t)a.tok.rows(), DBG_LOAD);
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            const bool ok = t < kTile && t < rows && fine;
            u[i] = load_quad<T>(a.u, a.u_stride, row0 + t, qc, left, ok, vec);
            dl[i] = load_quad<T>(a.delta, a.delta_stride, row0 + t, qc, left, ok, vec);
            if (!ENDS && a.z) z[i] = load_quad<T>(a.z, a.z_stride, row0 + t, qc, left, ok, vec);
        }
        vb.load(a.B, a.B_stride, row0, fine ? rows : 0, k.group, a.N);
        if (!ENDS) vc.load(a.C, a.C_stride, row0, fine ? rows : 0, k.group, a.N);
    };
    fetch(0);
    float total[4] = {};
    const long long tile0 = k.tiles0(a) + p.begin / kTile;
    for (int t0 = 0; t0 < p.len; t0 += kTile) {
        const int rows = min(kTile, p.len - t0);
        Vec<T, 4> cu[S::kPer], cz[S::kPer];
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            cu[i] = u[i];
            cz[i] = z[i];
            if (t >= kTile) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float d = dl[i][e] + bias[e];
                if (a.softplus) d = softplus(d);
                if (t >= rows) d = 0.f;  // nothing decays and nothing comes in behind the end
                const float x = d * u[i][e];
                if (ENDS) total[e] += d;
                sdx[t][4 * q + e] = make_float4(d, d, x, x);
            }
        }
        vb.put(sB);
        if (!ENDS) vc.put(sC);
        fetch(t0 + kTile);
        __syncthreads();
        if (!ENDS && a.saved && in) {
            const size_t at = ((size_t)(tile0 + t0 / kTile) * a.D + ch) * NP + n0;
            if (dbg_ok(a.dbg, at + 3, a.saved_floats, DBG_STORE)) *(float4 *)(a.saved + at) = one(h);
        }
#pragma unroll
        for (int tb = 0; tb < kTile; tb += 4) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 dx = sdx[tb + j][c];
                const Four Bv = four(*(const float4 *)&sB[tb + j][n0]);
                h = fma(decay(make_float2(dx.x, dx.y), A2), h, mul(make_float2(dx.z, dx.w), Bv));
                if (!ENDS) y[j] = dot(h, four(*(const float4 *)&sC[tb + j][n0]));
            }
            if (!ENDS) {
                scatter_sum<S::L, 1>(y, tid);
                using W = Share<S::L>;
                if (W::mine(part)) {
#pragma unroll
                    for (int j = 0; j < W::kCount; ++j) sy[tb + W::first(part) + j][c] = y[j];
                }
            }
        }
        __syncthreads();
        if (!ENDS) {
#pragma unroll
            for (int i = 0; i < S::kPer; ++i) {
                const int t = qt + i * kStep;
                const long long row = p.row0 + p.begin + t0 + t;
                if (t >= rows || !dbg_ok(a.dbg, (size_t)row, (size_t)a.tok.rows(), DBG_STORE)) continue;
                const float4 s = *(const float4 *)&sy[t][4 * q];
                const float sum[4] = {s.x, s.y, s.z, s.w};
                Vec<T, 4> out;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y = fmaf(skip[e], cu[i][e], sum[e]);
                    if (a.z) {
                        const float g = cz[i][e];
                        y *= g * sigmoid(g);
                    }
                    out.v[e] = from_f32<T>(y);
                }
                store_quad(a.y, a.y_stride, row, qc, left, out, vec);
            }
        }
    }
    if (ENDS) {
        const size_t at = (size_t)k.slot * a.D;
        if (in && dbg_ok(a.dbg, (at + ch) * NP + NP - 1, a.segment_floats, DBG_STORE))
            *(float4 *)(a.ends + (at + ch) * NP + n0) = one(h);
        // step sizes: the threads of a quad each have some tokens' sums
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (qt < kTile) sy[qt][4 * q + e] = total[e];
        __syncthreads();
        if (tid < k.channels) {
            float s = 0.f;
            for (int t = 0; t < min(kTile, kStep); ++t) s += sy[t][tid];
            a.sums[at + k.c0 + tid] = s;
        }
    } else if (a.final && in && p.begin + p.len == p.total) {
        if (dbg_ok(a.dbg, (size_t)p.seq, (size_t)a.tok.num_seqs, DBG_STORE))
            store_states(a.final, (size_t)p.seq * a.D + ch, n0, a.N, h);
    }
}

template <typename T, int NP> cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    const int per = a.D / a.G, nb = (per + Shape<NP>::CH - 1) / Shape<NP>::CH;
    const bool vec = per % 4 == 0 && vec_ok(a, a.u, a.u_stride) && vec_ok(a, a.delta, a.delta_stride) &&
                     vec_ok(a, a.z, a.z_stride) && vec_ok(a, a.y, a.y_stride);
    const unsigned grid = (unsigned)(a.tok.pieces(a.segment) * nb * a.G);
    if (a.ends) {
        const cudaError_t e = launch_early(kda_scan_fwd_kernel<T, NP, true>, grid, kThreads, 0, stream, a, nb, vec);
        if (e != cudaSuccess) return e;
    }
    return launch_early(kda_scan_fwd_kernel<T, NP, false>, grid, kThreads, 0, stream, a, nb, vec);
}

template <typename T> cudaError_t pick(const ScanArgs &a, cudaStream_t stream) {
    switch (scan_padded(a.N)) {
        case 4: return launch<T, 4>(a, stream);
        case 8: return launch<T, 8>(a, stream);
        case 16: return launch<T, 16>(a, stream);
        case 32: return launch<T, 32>(a, stream);
    }
    return launch<T, 64>(a, stream);
}

}  // namespace
}  // namespace scan

// Tokens of a segment: whole sequences where they fill the card (some four CTAs a multiprocessor),
// otherwise so many segments that they do.
int scan_segment(const Tokens &tok, int D, int N, int G, bool back) {
    const long long blocks = scan_blocks(D, N, G), want = 4 * kSMs;
    const long long rows = tok.rows(), longest = tok.cu_seqlens ? rows : tok.T;
    long long cuts = want / blocks;  // segments of all tokens together
    if (cuts < 1) cuts = 1;
    const long long whole = (longest + kScanTile - 1) / kScanTile * kScanTile;
    if (!tok.cu_seqlens && tok.num_seqs * blocks * 2 > want) return (int)(whole ? whole : kScanTile);
    long long seg = (rows / cuts + kScanTile - 1) / kScanTile * kScanTile;
    if (seg < 8 * kScanTile) seg = 8 * kScanTile;
    return (int)(seg < whole ? seg : whole ? whole : kScanTile);
}

cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return scan::pick<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return scan::pick<__half>(a, stream);
    return scan::pick<float>(a, stream);
}

}  // namespace kda
