// Selective scan, backward (kda_scan.cuh has the forward's formulas).  With p_t = exp(D_t A) h_{t-1}
// and dy' = dy silu(z), walking back from a sequence's end,
//   g_t = C_t dy'_t + exp(D_{t+1} A) g_{t+1},
//   dC_t = sum_d dy'_t h_t,   dB_t = sum_d g_t D_t u_t,   dA = sum_t g_t p_t D_t,
//   du_t = D_t sum_n g_t B_t + skip dy'_t,   dD_t = u_t sum_n g_t B_t + sum_n g_t p_t A,
//   ddelta_t = dD_t softplus'(delta_t + delta_bias),   dskip = sum_t dy'_t u_t,
//   dz_t = dy_t (sum_n C_t h_t + skip u_t) silu'(z_t).
// The states come again from the ones that the forward left in front of every 16 tokens: half a
// tile at a time, so that eight tokens' p stay in registers (h is p + D u B, without a difference
// that would lose small p).  Sums over a channel's states as in the forward; dB and dC are summed
// over a warp's channels by lanes that each end with one of their 2 NP values, over the CTA's warps
// in shared memory and over the CTAs by a second kernel, always in the same order.
#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

constexpr int kHalf = 8;

template <int NP> struct Smem {
    using S = Shape<NP>;
    float4 dx[kTile][S::CH];       // step size twice, step size times input twice
    float g[kTile][S::CH];         // dy'
    float B[kTile][NP], C[kTile][NP];
    float sum[3][kTile][S::kRow];  // over a channel's states: g B, g p A, C h
    float bc[kThreads / 32][kHalf][2 * NP];
};

// The first pass over segments: what each one's tokens leave of g in front of it.
template <typename T, int NP>
__global__ void __launch_bounds__(kThreads) kda_scan_bwd_ends_kernel(const ScanArgs a, int nb, bool vec) {
    wait_for_previous();
    using S = Shape<NP>;
    __shared__ float2 sdg[kTile][S::CH];
    __shared__ __align__(16) float sC[kTile][NP], st[kTile][S::kRow];
    const int tid = threadIdx.x, c = tid / S::L, n0 = 4 * (tid % S::L);
    const Block<NP> k(a, nb);
    const Piece &p = k.p;
    if (p.len < 0 || p.begin == 0) return;
    const bool in = c < k.channels;
    const size_t ch = (size_t)k.c0 + c;
    const Four A2 = scaled(load_states(a.A, ch, n0, a.N, in), kLog2e);
    Four g = {both(0.f), both(0.f)};
    const int q = tid % S::kQuads, qt = tid / S::kQuads, qc = k.c0 + 4 * q, left = k.channels - 4 * q;
    constexpr int kStep = kThreads / S::kQuads;
    float total[4] = {};
    Vec<T, 4> dl[S::kPer], dy[S::kPer], z[S::kPer];
    Vectors<T, NP> vc;
    auto fetch = [&](int t0) {
        const int rows = t0 < 0 ? 0 : p.len - t0;
        const long long row0 = p.row0 + p.begin + t0;
        const bool fine = rows <= 0 || dbg_ok(a.dbg, (size_t)(row0 + min(rows, kTile) - 1), (size_t)a.tok.rows(), DBG_LOAD);
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            const bool ok = t < kTile && t < rows && fine;
            dl[i] = load_quad<T>(a.delta, a.delta_stride, row0 + t, qc, left, ok, vec);
            dy[i] = load_quad<T>(a.dy, a.dy_stride, row0 + t, qc, left, ok, vec);
            if (a.z) z[i] = load_quad<T>(a.z, a.z_stride, row0 + t, qc, left, ok, vec);
        }
        vc.load(a.C, a.C_stride, row0, fine ? rows : 0, k.group, a.N);
    };
    const int last = (p.len - 1) / kTile * kTile;
    fetch(last);
    for (int t0 = last; t0 >= 0; t0 -= kTile) {
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            if (t >= kTile) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float d = dl[i][e] + (a.delta_bias && e < left ? a.delta_bias[qc + e] : 0.f);
                if (a.softplus) d = softplus(d);
                if (t >= p.len - t0) d = 0.f;
                float y = dy[i][e];
                if (a.z) y *= z[i][e] * sigmoid(z[i][e]);
                total[e] += d;
                sdg[t][4 * q + e] = make_float2(d, y);
            }
        }
        vc.put(sC);
        fetch(t0 - kTile);
        __syncthreads();
#pragma unroll
        for (int t = kTile - 1; t >= 0; --t) {
            const float2 x = sdg[t][c];
            g = mul(fma(both(x.y), four(*(const float4 *)&sC[t][n0]), g), decay(both(x.x), A2));
        }
        __syncthreads();
    }
    const size_t at = (size_t)k.slot * a.D;
    if (in && dbg_ok(a.dbg, (at + ch) * NP + NP - 1, a.segment_floats, DBG_STORE))
        *(float4 *)(a.ends + (at + ch) * NP + n0) = one(g);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (qt < kTile) st[qt][4 * q + e] = total[e];
    __syncthreads();
    if (tid < k.channels) {
        float s = 0.f;
        for (int t = 0; t < min(kTile, kStep); ++t) s += st[t][tid];
        a.sums[at + k.c0 + tid] = s;
    }
}

template <typename T, int NP>
__global__ void __launch_bounds__(kThreads, 4) kda_scan_bwd_kernel(const ScanArgs a, int nb, bool vec) {
    wait_for_previous();
    using S = Shape<NP>;
    extern __shared__ __align__(16) char raw[];
    Smem<NP> &s = *reinterpret_cast<Smem<NP> *>(raw);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const int c = tid / S::L, part = tid % S::L, n0 = 4 * part;
    const Block<NP> k(a, nb);
    const Piece &p = k.p;
    const bool in = c < k.channels;
    const size_t ch = (size_t)k.c0 + c;
    const Four A2 = scaled(load_states(a.A, ch, n0, a.N, in), kLog2e);
    Four carry = {both(0.f), both(0.f)}, dA = carry;
    if (p.len >= 0 && in) {  // from the segments behind this one
        carry = load_states(a.d_final, (size_t)p.seq * a.D + ch, n0, a.N, a.d_final);
        const int behind = (p.total + a.segment - 1) / a.segment - 1 - p.index;
        for (int j = k.slot + behind; j > k.slot; --j) {
            const size_t at = (size_t)j * a.D + ch;
            if (!dbg_ok(a.dbg, at * NP + NP - 1, a.segment_floats, DBG_LOAD)) break;
            carry = fma(decay(both(a.sums[at]), A2), carry, four(*(const float4 *)(a.ends + at * NP + n0)));
        }
    }
    const int q = tid % S::kQuads, qt = tid / S::kQuads, qc = k.c0 + 4 * q, left = k.channels - 4 * q;
    constexpr int kStep = kThreads / S::kQuads;
    float bias[4], skip[4], dskip[4] = {}, dbias[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = a.delta_bias && i < left ? a.delta_bias[qc + i] : 0.f;
        skip[i] = a.skip && i < left ? a.skip[qc + i] : 0.f;
    }
    const long long tile0 = k.tiles0(a) + p.begin / kTile;
    const int first = p.len > 0 ? (p.len - 1) / kTile * kTile : -1;
    for (int t0 = first; t0 >= 0; t0 -= kTile) {
        const int rows = min(kTile, p.len - t0);
        const long long row0 = p.row0 + p.begin + t0;
        const bool fine = dbg_ok(a.dbg, (size_t)(row0 + rows - 1), (size_t)a.tok.rows(), DBG_LOAD | DBG_STORE);
        Vec<T, 4> u[S::kPer], dl[S::kPer], z[S::kPer], dy[S::kPer];
        Vectors<T, NP> vb, vc;
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            const bool ok = t < rows && fine;
            u[i] = load_quad<T>(a.u, a.u_stride, row0 + t, qc, left, ok, vec);
            dl[i] = load_quad<T>(a.delta, a.delta_stride, row0 + t, qc, left, ok, vec);
            dy[i] = load_quad<T>(a.dy, a.dy_stride, row0 + t, qc, left, ok, vec);
            if (a.z) z[i] = load_quad<T>(a.z, a.z_stride, row0 + t, qc, left, ok, vec);
        }
        vb.load(a.B, a.B_stride, row0, fine ? rows : 0, k.group, a.N);
        vc.load(a.C, a.C_stride, row0, fine ? rows : 0, k.group, a.N);
        Four h0 = {both(0.f), both(0.f)};
        {
            const size_t at = ((size_t)(tile0 + t0 / kTile) * a.D + ch) * NP + n0;
            if (in && dbg_ok(a.dbg, at + 3, a.saved_floats, DBG_LOAD)) h0 = four(*(const float4 *)(a.saved + at));
        }
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            if (t >= kTile) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float d = dl[i][e] + bias[e];
                if (a.softplus) d = softplus(d);
                if (t >= rows) d = 0.f;
                const float x = d * u[i][e];
                s.dx[t][4 * q + e] = make_float4(d, d, x, x);
                s.g[t][4 * q + e] = a.z ? dy[i][e] * z[i][e] * sigmoid(z[i][e]) : dy[i][e];
            }
        }
        vb.put(s.B);
        vc.put(s.C);
        __syncthreads();
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
            Four h = h0, pr[kHalf];
            if (half == 1) {
#pragma unroll
                for (int t = 0; t < kHalf; ++t) {
                    const float4 dx = s.dx[t][c];
                    h = fma(decay(make_float2(dx.x, dx.y), A2), h,
                            mul(make_float2(dx.z, dx.w), four(*(const float4 *)&s.B[t][n0])));
                }
            }
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const int t = half * kHalf + j;
                const float4 dx = s.dx[t][c];
                pr[j] = mul(decay(make_float2(dx.x, dx.y), A2), h);
                h = fma(make_float2(dx.z, dx.w), four(*(const float4 *)&s.B[t][n0]), pr[j]);
            }
#pragma unroll
            for (int jb = kHalf - 4; jb >= 0; jb -= 4) {
                float gb[4], gpa[4], y[4];
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    const int j = jb + i, t = half * kHalf + j;
                    const float4 dx = s.dx[t][c];
                    const float2 dd = make_float2(dx.x, dx.y), xx = make_float2(dx.z, dx.w);
                    const float2 gg = both(s.g[t][c]);
                    const Four Bv = four(*(const float4 *)&s.B[t][n0]), Cv = four(*(const float4 *)&s.C[t][n0]);
                    const Four g = fma(gg, Cv, carry), hj = fma(xx, Bv, pr[j]), gp = mul(g, pr[j]);
                    gb[i] = dot(g, Bv);
                    gpa[i] = dot(gp, A2);
                    y[i] = dot(hj, Cv);
                    dA = fma(dd, gp, dA);
                    carry = mul(g, decay(dd, A2));
                    const Four b = mul(xx, g), cc = mul(gg, hj);
                    float v[8] = {b.lo.x, b.lo.y, b.hi.x, b.hi.y, cc.lo.x, cc.lo.y, cc.hi.x, cc.hi.y};
                    constexpr int CW = 32 / S::L, kLeft = CW < 8 ? 8 / CW : 1;
                    scatter_sum<CW, S::L>(v, lane);
                    const int cl = lane / S::L;  // channel in the warp
                    if (CW <= 8 || cl % (CW / 8 > 0 ? CW / 8 : 1) == 0) {
                        const int at = CW < 8 ? cl * kLeft : cl / (CW / 8 > 0 ? CW / 8 : 1);
#pragma unroll
                        for (int x = 0; x < kLeft; ++x) {
                            const int idx = at + x;  // 0..3: dB, 4..7: dC of the lane's states
                            s.bc[warp][j][(idx < 4 ? 0 : NP) + n0 + (idx & 3)] = v[x];
                        }
                    }
                }
                scatter_sum<S::L, 1>(gb, tid);
                scatter_sum<S::L, 1>(gpa, tid);
                scatter_sum<S::L, 1>(y, tid);
                using W = Share<S::L>;
                if (W::mine(part)) {
#pragma unroll
                    for (int i = 0; i < W::kCount; ++i) {
                        const int t = half * kHalf + jb + W::first(part) + i;
                        s.sum[0][t][c] = gb[i];
                        s.sum[1][t][c] = gpa[i];
                        s.sum[2][t][c] = y[i];
                    }
                }
            }
            __syncthreads();
            for (int e = tid; e < kHalf * 2 * NP; e += kThreads) {
                const int j = e / (2 * NP), x = e % (2 * NP), t = half * kHalf + j;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) v += s.bc[w][j][x];
                if (t < rows && fine)
                    a.part_bc[(((size_t)k.blk * a.tok.rows() + row0 + t) * a.G + k.group) * 2 * NP + x] = v;
            }
            if (half == 1) __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            if (t >= rows || !fine) continue;
            Vec<T, 4> du, dd, dz;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int cc = 4 * q + e;
                const float gb = s.sum[0][t][cc], gpa = s.sum[1][t][cc] * kLn2, y = s.sum[2][t][cc];
                const float d = s.dx[t][cc].x, g = s.g[t][cc], uu = u[i][e];
                du.v[e] = from_f32<T>(fmaf(d, gb, skip[e] * g));
                float x = fmaf(uu, gb, gpa);
                if (a.softplus) x *= sigmoid(dl[i][e] + bias[e]);
                dd.v[e] = from_f32<T>(x);
                dbias[e] += x;
                dskip[e] = fmaf(g, uu, dskip[e]);
                if (a.z) {
                    const float zz = z[i][e];
                    dz.v[e] = from_f32<T>(dy[i][e] * fmaf(skip[e], uu, y) * silu_slope(zz, sigmoid(zz)));
                }
            }
            store_quad(a.du, a.du_stride, row0 + t, qc, left, du, vec);
            store_quad(a.ddelta, a.ddelta_stride, row0 + t, qc, left, dd, vec);
            if (a.z) store_quad(a.dz, a.dz_stride, row0 + t, qc, left, dz, vec);
        }
        __syncthreads();
    }
    if (p.len >= 0 && p.begin == 0 && in && a.d_initial && dbg_ok(a.dbg, (size_t)p.seq, (size_t)a.tok.num_seqs, DBG_STORE))
        store_states(a.d_initial, (size_t)p.seq * a.D + ch, n0, a.N, carry);
    // the parameters' sums over this segment
    const size_t at = (size_t)k.slot * a.D;
    if (in && dbg_ok(a.dbg, (at + ch) * NP + NP - 1, a.segment_floats, DBG_STORE))
        *(float4 *)(a.part_A + (at + ch) * NP + n0) = one(dA);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (qt < kTile) {
            s.sum[0][qt][4 * q + e] = dskip[e];
            s.sum[1][qt][4 * q + e] = dbias[e];
        }
    __syncthreads();
    if (tid < k.channels) {
        float x = 0.f, y = 0.f;
        for (int t = 0; t < min(kTile, kStep); ++t) {
            x += s.sum[0][t][tid];
            y += s.sum[1][t][tid];
        }
        a.part_D[2 * at + k.c0 + tid] = x;
        a.part_D[2 * at + a.D + k.c0 + tid] = y;
    }
}

// dB and dC of the tokens that are in a sequence: sums over the blocks of channels, in order.
template <typename T>
__global__ void __launch_bounds__(256) kda_scan_sum_bc_kernel(const ScanArgs a, int nb, int np) {
    wait_for_previous();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, wide = (long long)a.G * 2 * np;
    const long long row = i / wide;
    const int rest = (int)(i - row * wide), group = rest / (2 * np), x = rest % (2 * np);
    if (row >= a.tok.rows()) return;
    if (a.tok.cu_seqlens && (row < a.tok.cu_seqlens[0] || row >= a.tok.cu_seqlens[a.tok.num_seqs])) return;
    const int n = x % np;
    if (n >= a.N) return;
    float s = 0.f;
    const size_t step = (size_t)a.tok.rows() * wide;
#pragma unroll 8
    for (int b = 0; b < nb; ++b) s += a.part_bc[b * step + i];
    ((T *)(x < np ? a.dB : a.dC))[((size_t)row * a.G + group) * a.N + n] = from_f32<T>(s);
}

// dA, dskip and ddelta_bias: sums over the segments, in order.
__global__ void __launch_bounds__(256) kda_scan_sum_params_kernel(const ScanArgs a, int slots, int np) {
    wait_for_previous();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, states = (long long)a.D * np;
    float s = 0.f;
    if (i < states) {
        const int n = (int)(i % np);
        if (n >= a.N) return;
#pragma unroll 4
        for (int j = 0; j < slots; ++j) s += a.part_A[j * states + i];
        a.dA[i / np * a.N + n] = s;
    } else if (i < states + 2 * a.D) {
        const int x = (int)(i - states);
#pragma unroll 4
        for (int j = 0; j < slots; ++j) s += a.part_D[(size_t)j * 2 * a.D + x];
        float *to = x < a.D ? a.dskip : a.ddelta_bias;
        if (to) to[x < a.D ? x : x - a.D] = s;
    }
}

template <typename T, int NP> cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    const int per = a.D / a.G, nb = (per + Shape<NP>::CH - 1) / Shape<NP>::CH;
    const bool vec = per % 4 == 0 && vec_ok(a, a.u, a.u_stride) && vec_ok(a, a.delta, a.delta_stride) &&
                     vec_ok(a, a.z, a.z_stride) && vec_ok(a, a.dy, a.dy_stride) &&
                     vec_ok(a, a.du, a.du_stride) && vec_ok(a, a.ddelta, a.ddelta_stride) &&
                     vec_ok(a, a.dz, a.dz_stride);
    const long long slots = a.tok.pieces(a.segment);
    const unsigned grid = (unsigned)(slots * nb * a.G);
    constexpr int kBytes = sizeof(Smem<NP>);
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = smem_limit_once(kda_scan_bwd_kernel<T, NP>, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    if (a.ends) {
        e = launch_early(kda_scan_bwd_ends_kernel<T, NP>, grid, kThreads, 0, stream, a, nb, vec);
        if (e != cudaSuccess) return e;
    }
    e = launch_early(kda_scan_bwd_kernel<T, NP>, grid, kThreads, kBytes, stream, a, nb, vec);
    if (e != cudaSuccess) return e;
    const long long bc = a.tok.rows() * a.G * 2 * NP;
    if (bc) {
        e = launch_early(kda_scan_sum_bc_kernel<T>, (unsigned)((bc + 255) / 256), 256, 0, stream, a, nb, NP);
        if (e != cudaSuccess) return e;
    }
    const long long params = (long long)a.D * (NP + 2);
    return launch_early(kda_scan_sum_params_kernel, (unsigned)((params + 255) / 256), 256, 0, stream, a,
                        (int)slots, NP);
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

cudaError_t launch_scan_bwd(const ScanArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return scan::pick<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return scan::pick<__half>(a, stream);
    return scan::pick<float>(a, stream);
}

}  // namespace kda
