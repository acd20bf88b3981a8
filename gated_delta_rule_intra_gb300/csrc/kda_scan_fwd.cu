// Selective scan, forward (kda_scan.cuh).
//
// A tile's three phases -- preparing the next tile, the scan of this one, finishing the one before --
// have buffers of their own, so that one barrier a tile joins them; inputs are asked for three
// tiles ahead.
//
// Bound by what a warp waits for (issue slots 54%, shared memory's data pipe 59%; two CTAs a
// multiprocessor take 478 us for 4096 tokens of 64 channels each, one alone 425): 256 us at B=4 T=2048
// D=4096 N=16 bf16 (256 CTAs; 240 where nothing is saved; fp32 288), where the bytes are 40 at a copy's rate
// and the exponentials 58; 32768 tokens 1250.  One
// channel a thread took 475 us, two without the order of states that lets their sums be shared 387.
#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

constexpr int kStages = 4;

template <typename T, int NP> struct Smem {
    using S = Shape<NP>;
    float d[2][S::CH * kTile], x[2][S::CH * kTile];  // step size, step size times input: place()
    float B[2][S::L][S::kVec], C[2][S::L][S::kVec];
    float y[2][kTile][S::kRow];                       // sums over a channel's states
    float2 raise[2][kThreads];                        // Raise, of each walking thread
    Vec<T, 8> raw[kStages][3][S::kPer][kThreads];     // u, delta, z: a slot of each thread
};

// ENDS: the first pass, which leaves the segments' ends.
template <typename T, int NP, bool ENDS>
__global__ void __launch_bounds__(2 * kThreads, 2) kda_scan_fwd_kernel(const ScanArgs a, int nb, int unit) {
    wait_for_previous();
    using S = Shape<NP>;
    extern __shared__ __align__(16) char smem[];
    using M = Smem<T, NP>;
    M &s = *reinterpret_cast<M *>(smem);
    const Block<NP> k(a, nb);
    const Piece &p = k.p;
    if (p.len < 0 || (ENDS && p.begin + p.len == p.total)) return;
    const int tiles = (p.len + kTile - 1) / kTile;
    const long long first = p.row0 + p.begin;
    const size_t seg = (size_t)k.slot * a.D;
    if (threadIdx.x < kThreads) {  // the scan
        const int tid = threadIdx.x, part = tid % S::L, n0 = 4 * part, turn = turn_of<NP>(tid);
        const int c[2] = {tid / S::L, tid / S::L + S::HC};
        uint64_t A2[2][4];
        float h[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bool in = c[j] < k.channels;
            const size_t ch = (size_t)k.c0 + c[j];
            const Four Aj = scaled(load_states(a.A, ch, n0, a.N, in, turn), kLog2e);
            Four hj = {both(0.f), both(0.f)};
            if (!ENDS && in) {
                const bool given = a.initial && in_bounds(a.dbg, (size_t)p.seq, (size_t)a.tok.num_seqs, DBG_LOAD);
                hj = load_states(a.initial, (size_t)p.seq * a.D + ch, n0, a.N, given, turn);
                for (int g = k.slot - p.index; g < k.slot; ++g) {
                    const size_t at = (size_t)g * a.D + ch;
                    if (!in_bounds(a.dbg, at * NP + NP - 1, a.segment_floats, DBG_LOAD) ||
                        !in_bounds(a.dbg, at, a.sum_floats, DBG_LOAD))
                        break;
                    hj = fma(decay(both(a.sums[at]), Aj, 0.f), hj, four(*(const float4 *)(a.ends + at * NP + n0)));
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                A2[j][n] = twice(Aj.get(n));
                h[j][n] = hj.get(n);
            }
        }
        const long long tile0 = k.tiles0(a) + p.begin / kTile;
        Phase phase(smem);
        if (tiles > 0) sync_all();
        for (int tile = 0; tile < tiles; ++tile) {
            const int b = tile & 1;
            phase.next();
            auto save = [&](int half) {  // the states in front of half a tile
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const size_t at = ((size_t)(2 * (tile0 + tile) + half) * a.D + k.c0 + c[j]) * NP + n0;
                    if (c[j] < k.channels && in_bounds(a.dbg, at + 3, a.saved_floats, DBG_STORE))
                        *(float4 *)(a.saved + at) = make_float4(h[j][0], h[j][1], h[j][2], h[j][3]);
                }
            };
            const uint32_t od = (uint32_t)((char *)s.d[b] - smem), ox = (uint32_t)((char *)s.x[b] - smem);
            uint32_t oB[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) oB[n] = (uint32_t)((char *)&s.B[b][part][(n ^ turn) * kTile] - smem);
            constexpr uint32_t toC = offsetof(M, C) - offsetof(M, B);
            const uint64_t raise = ENDS ? 0 : phase.load_pair((uint32_t)((char *)&s.raise[b][tid] - smem));
#pragma unroll
            for (int g = 0; g < kTile / 4; ++g) {
                if (!ENDS && a.saved && g % 2 == 0) save(g / 2);
                float2 B[4][2], C[4][2];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    phase.load4(oB[n] + 16 * g, B[n]);
                    if (!ENDS) phase.load4(oB[n] + toC + 16 * g, C[n]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float2 d[2], x[2];
                    phase.load4(od + 4 * place(c[j], g), d);
                    phase.load4(ox + 4 * place(c[j], g), x);
                    float y[4];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        float2 sum;
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const float2 e = ENDS ? exponent(d[t], A2[j][n]) : fma2(d[t], A2[j][n], raise);
                            const float2 in = mul2(x[t], B[n][t]);
                            float2 hh;
                            hh.x = fmaf(ex2(e.x), h[j][n], in.x);
                            hh.y = fmaf(ex2(e.y), hh.x, in.y);
                            h[j][n] = hh.y;
                            if (!ENDS) sum = n ? fma2(C[n][t], hh, sum) : mul2(C[n][t], hh);
                        }
                        y[2 * t] = sum.x;
                        y[2 * t + 1] = sum.y;
                    }
                    if (!ENDS) {
                        scatter_sum<S::L, 1>(y, tid);
                        using W = Share<S::L>;
                        if (W::mine(part)) {
#pragma unroll
                            for (int i = 0; i < W::kCount; ++i) s.y[b][4 * g + W::first(part) + i][c[j]] = y[i];
                        }
                    }
                }
            }
            sync_all();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const size_t ch = (size_t)k.c0 + c[j];
            if (c[j] >= k.channels) continue;
            if (ENDS && in_bounds(a.dbg, (seg + ch) * NP + NP - 1, a.segment_floats, DBG_STORE))
                *(float4 *)(a.ends + (seg + ch) * NP + n0) = make_float4(h[j][0], h[j][1], h[j][2], h[j][3]);
            if (!ENDS && a.final && p.begin + p.len == p.total &&
                in_bounds(a.dbg, (size_t)p.seq, (size_t)a.tok.num_seqs, DBG_STORE))
                store_states(a.final, (size_t)p.seq * a.D + ch, n0, a.N,
                             four(make_float4(h[j][0], h[j][1], h[j][2], h[j][3])), turn);
        }
        return;
    }
    // this thread's chunks of a tile: tokens qt + i kStep, channels 8 q ..
    const int tid = threadIdx.x - kThreads;
    const int q = tid % S::kChunks, qt = tid / S::kChunks, qc = k.c0 + 8 * q, left = k.channels - 8 * q;
    constexpr int kStep = kThreads / S::kChunks;
    float2 bias[4], skip[4], total[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        auto param = [&](const float *v, int i) { return v && i < left ? v[qc + i] : 0.f; };
        bias[e] = make_float2(param(a.delta_bias, 2 * e), param(a.delta_bias, 2 * e + 1));
        skip[e] = make_float2(param(a.skip, 2 * e), param(a.skip, 2 * e + 1));
    }
    auto rows_of = [&](int tile) { return p.len - tile * kTile; };
    auto fine = [&](int tile) {
        const int rows = rows_of(tile);
        return rows <= 0 || in_bounds(a.dbg, (size_t)(first + tile * kTile + min(rows, kTile) - 1), (size_t)a.tok.rows(), DBG_LOAD);
    };
    auto fetch = [&](int tile) {
        const int rows = fine(tile) ? rows_of(tile) : 0;
        auto &raw = s.raw[tile % kStages];
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            const bool ok = t < kTile && t < rows;
            const long long row = ok ? first + tile * kTile + t : 0;
            fetch_chunk<T>(&raw[0][i][tid], a.u, (const T *)a.u + row * a.u_stride + qc, left, ok, unit);
            fetch_chunk<T>(&raw[1][i][tid], a.delta, (const T *)a.delta + row * a.delta_stride + qc, left, ok, unit);
            if (!ENDS && a.z) fetch_chunk<T>(&raw[2][i][tid], a.z, (const T *)a.z + row * a.z_stride + qc, left, ok, unit);
        }
        cp_async_commit();
    };
    Vectors<T, NP> vb, vc;
    const Raise<NP> raise(a, k.c0, k.channels, tid);
    auto vectors = [&](int tile) {
        const int rows = fine(tile) ? rows_of(tile) : 0;
        vb.load(tid, a.B, a.B_stride, first + tile * kTile, rows, k.group, a.N);
        if (!ENDS) vc.load(tid, a.C, a.C_stride, first + tile * kTile, rows, k.group, a.N);
    };
    auto prepare = [&](int tile) {
        const int rows = rows_of(tile), b = tile & 1;
        auto &raw = s.raw[tile % kStages];
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            if (t >= kTile) continue;
            const Vec<T, 8> u = raw[0][i][tid], dl = raw[1][i][tid];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 d = add2(pair(dl, e), bias[e]);
                if (a.softplus) d = softplus(d);
                if (t >= rows) d = both(0.f);  // nothing decays and nothing comes in behind the end
                const float2 x = mul2(d, pair(u, e));
                if (ENDS) total[e] = add2(total[e], d);
                const int at = place(8 * q + 2 * e, t >> 2) + (t & 3);
                s.d[b][at] = d.x;
                s.d[b][at + kTile] = d.y;
                s.x[b][at] = x.x;
                s.x[b][at + kTile] = x.y;
            }
        }
        vb.put(tid, s.B[b]);
        if (!ENDS) {
            vc.put(tid, s.C[b]);
            s.raise[b][tid] = tile > 0 ? raise.next(s.d[b ^ 1]) : both(kQuick);
        }
    };
    const bool quads = a.D / a.G % 4 == 0;  // blocks of channels begin on four
    auto finish = [&](int tile) {
        const int rows = rows_of(tile), b = tile & 1;
        auto &raw = s.raw[tile % kStages];
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int t = qt + i * kStep;
            const long long row = first + tile * kTile + t;
            if (t >= kTile || t >= rows || !in_bounds(a.dbg, (size_t)row, (size_t)a.tok.rows(), DBG_STORE)) continue;
            const float4 lo = *(const float4 *)&s.y[b][t][8 * q], hi = *(const float4 *)&s.y[b][t][8 * q + 4];
            const float2 sum[4] = {make_float2(lo.x, lo.y), make_float2(lo.z, lo.w), make_float2(hi.x, hi.y),
                                   make_float2(hi.z, hi.w)};
            const Vec<T, 8> u = raw[0][i][tid];
            Vec<T, 8> z, out;
            float2 open[4];
            if (a.z) z = raw[2][i][tid];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 y = fma2(skip[e], pair(u, e), sum[e]);
                if (a.z) {
                    const float2 g = pair(z, e);
                    open[e] = y;
                    y = mul2(y, mul2(g, sigmoid2(g)));
                }
                put_pair(out, e, y);
            }
            if (a.open && in_bounds(a.dbg, (size_t)(open_row(a, row) - a.open) + qc + min(left, 8) - 1, a.open_floats, DBG_STORE)) {
                // what the gate multiplies, for the gate's gradient
                float *at = open_row(a, row) + qc;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 l = open[2 * h], r = open[2 * h + 1];
                    if (quads && 4 * h < left) *(float4 *)(at + 4 * h) = make_float4(l.x, l.y, r.x, r.y);
                    if (!quads) {
                        const float v[4] = {l.x, l.y, r.x, r.y};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (4 * h + j < left) at[4 * h + j] = v[j];
                    }
                }
            }
            store_chunk(a.y, a.y_stride, row, qc, left, out, unit);
        }
    };
    if (tiles > 0) {
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i);
        vectors(0);
        cp_async_wait_newest<kStages - 2>();
        prepare(0);
        vectors(1);
        sync_all();
    }
    for (int tile = 0; tile < tiles; ++tile) {
        if (tile + 1 < tiles) {
            cp_async_wait_newest<1>();
            prepare(tile + 1);
            vectors(tile + 2);
        }
        if (!ENDS && tile > 0) finish(tile - 1);
        fetch(tile + kStages - 1);
        sync_all();
    }
    if (!ENDS && tiles > 0) finish(tiles - 1);
    if (ENDS) {  // step sizes: the threads of a chunk's channels each have some tokens' sums
        auto &sum = s.y[0];
        if (qt < kTile) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[qt][8 * q + 2 * e] = total[e].x;
                sum[qt][8 * q + 2 * e + 1] = total[e].y;
            }
        }
        sync_half();
        if (tid < k.channels) {
            float x = 0.f;
            for (int t = 0; t < min(kTile, kStep); ++t) x += sum[t][tid];
            if (in_bounds(a.dbg, seg + k.c0 + tid, a.sum_floats, DBG_STORE)) a.sums[seg + k.c0 + tid] = x;
        }
    }
    cp_async_wait_newest<0>();
}

template <typename T, int NP> cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    const int per = a.D / a.G, nb = (per + Shape<NP>::CH - 1) / Shape<NP>::CH;
    Unit u(a);
    u.add(a.u, a.u_stride);
    u.add(a.delta, a.delta_stride);
    u.add(a.z, a.z_stride);
    u.add(a.y, a.y_stride);
    const unsigned grid = (unsigned)(a.tok.pieces(a.segment) * nb * a.G);
    constexpr int kBytes = sizeof(Smem<T, NP>);
    static_assert(kBytes <= 227 * 1024, "");
    static volatile int done[2][kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = smem_limit_once(kda_scan_fwd_kernel<T, NP, true>, kBytes, dev, done[0]);
    if (e == cudaSuccess) e = smem_limit_once(kda_scan_fwd_kernel<T, NP, false>, kBytes, dev, done[1]);
    if (e != cudaSuccess) return e;
    if (a.ends) {
        e = launch_early(kda_scan_fwd_kernel<T, NP, true>, grid, 2 * kThreads, kBytes, stream, a, nb, u.unit);
        if (e != cudaSuccess) return e;
    }
    return launch_early(kda_scan_fwd_kernel<T, NP, false>, grid, 2 * kThreads, kBytes, stream, a, nb, u.unit);
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

// Tokens of a segment.  Sequences of one length are cut where the rounds of two CTAs a multiprocessor
// (in tokens that one walks, and 32 for its start) and the first pass, which costs 0.7 of the second
// forward and 0.35 backward, take less than walking them whole; a CTA that is alone on its
// multiprocessor takes nine tenths of the time of two.  4096 tokens, 16 states, forward and backward, us:
//   64 chains of 64 channels: 9 segments 184 and 442, whole 331 and 968; 128: 7 segments 339 and 813,
//   whole 425 and 1332; 192: 3 segments 506 and 1220, whole 478 and 1432; 256: 677 and 1612, 477 and 1438.
// Packed ones, whose lengths the host does not know, take four segments a multiprocessor in all (9467 tokens
// in 9 sequences, 16 chains: 120 and 285; two 118 and 293, six 129 and 304).
int scan_segment(const Tokens &tok, int D, int N, int G, bool back) {
    const long long blocks = scan_blocks(D, N, G), chains = tok.num_seqs * blocks, slots = 2 * kSMs;
    auto tiles = [](long long tokens) { return (tokens + kScanTile - 1) / kScanTile * kScanTile; };
    const long long whole = tok.T ? tiles(tok.T) : kScanTile, least = 8 * kScanTile;
    long long best = whole;
    if (tok.cu_seqlens) {
        const long long cuts = 2 * slots / blocks, seg = tiles(tok.T / (cuts > 1 ? cuts : 1));
        best = seg < least ? least : seg;
    } else {
        long long cost = (chains + slots - 1) / slots * (whole + 32) * (chains <= kSMs ? 18 : 20);
        for (int rounds = 1; rounds <= 8; ++rounds) {
            const long long n = rounds * slots / chains, even = n > 1 ? tiles((tok.T + n - 1) / n) : whole;
            const long long seg = even < least ? least : even, c = rounds * (seg + 32) * (back ? 27 : 34);
            if (seg < whole && c < cost) {
                cost = c;
                best = seg;
            }
        }
    }
    return (int)(best < whole ? best : whole);
}

cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t stream) {
    if (a.dtype == TYPE_BF16) return scan::pick<__nv_bfloat16>(a, stream);
    if (a.dtype == TYPE_FP16) return scan::pick<__half>(a, stream);
    return scan::pick<float>(a, stream);
}

}  // namespace kda
