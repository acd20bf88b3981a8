// Selective scan, backward (kda_scan.cuh has the forward's formulas).  With p_t = exp(D_t A) h_{t-1}
// and dy' = dy silu(z), walking back from a sequence's end,
//   g_t = C_t dy'_t + exp(D_{t+1} A) g_{t+1},
//   dC_t = sum_d dy'_t h_t,   dB_t = sum_d g_t D_t u_t,   dA = sum_t g_t p_t D_t,
//   du_t = D_t sum_n g_t B_t + skip dy'_t,   dD_t = u_t sum_n g_t B_t + sum_n g_t p_t A,
//   ddelta_t = dD_t softplus'(delta_t + delta_bias),   dskip = sum_t dy'_t u_t,
//   dz_t = dy_t (sum_n C_t h_t + skip u_t) silu'(z_t).
// The states come again from the ones that the forward left in front of every eight tokens, whose p
// stay in registers (h is p + D u B, without a difference that would lose small p); so does what the
// gate multiplies.  (Checkpoints at every 16 tokens would halve their memory; the first eight would
// then be walked twice, 8% of the instructions.)  Sums over a channel's states as in the forward; dB and dC are summed
// over a thread's two channels, over a warp's by lanes that each end with one of the 8 values of
// four states, over the CTA's warps in shared memory and over the CTAs by a second kernel,
// always in the same order.
//
// Bound by what a warp waits for (issue slots 54%, shared memory's data pipe 63%): 726 us (fp32 979) at B=4 T=2048
// D=4096 N=16 bf16, where the bytes are 79 at a copy's rate and the exponentials 115.  With the gate's
// factor computed again from the states instead of read it took 954 us (the forward leaves it unrounded:
// 16 bits would save 8 us both ways and make dz's error 1.4 times its rounding), with both halves' registers
// alike 1038.
#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

constexpr int kHalf = 8, kWarps = kThreads / 32, kStages = 3;

// Registers: as many as a launch of two CTAs a multiprocessor has, moved to the half that walks.
constexpr int kLaunchRegs = 128, kWalkRegs = 168, kOtherRegs = 88;
static_assert(kWalkRegs + kOtherRegs == 2 * kLaunchRegs, "");

template <typename T, int NP, bool ENDS> struct Smem {
    using S = Shape<NP>;
    static constexpr int kSum = kTile * S::kRow + 16;
    float d[2][S::CH * kTile], x[2][S::CH * kTile], g[2][S::CH * kTile];  // D, D u, dy': place()
    float B[2][S::L][S::kVec], C[2][S::L][S::kVec];
    float sum[ENDS ? 1 : 2][2][kSum];  // over a channel's states: g B, g p A, [kTile][kRow] each
    float bc[ENDS ? 1 : 2][kWarps][kTile][2 * NP];
    float4 h[ENDS ? 1 : 2][2][2][kThreads];        // the states in front of half a tile: each thread's own
    float param[2][S::CH];                         // delta_bias, skip
    Vec<T, 8> raw[kStages][4][S::kPer][kThreads];  // u, delta, dy, z: a slot of each thread
};

// ENDS: the first pass over segments, which leaves what each one's tokens make of g in front of it.
template <typename T, int NP, bool ENDS>
__global__ void __launch_bounds__(2 * kThreads, 2) kda_scan_bwd_kernel(const ScanArgs a, int nb, int unit) {
    wait_for_previous();
    using S = Shape<NP>;
    using M = Smem<T, NP, ENDS>;
    extern __shared__ __align__(16) char smem[];
    M &s = *reinterpret_cast<M *>(smem);
    const Block<NP> k(a, nb);
    const Piece &p = k.p;
    if (ENDS && (p.len < 0 || p.begin == 0)) return;
    // tiles are taken from the last to the first: step i is tile tiles - 1 - i
    const int tiles = p.len > 0 ? (p.len + kTile - 1) / kTile : 0;
    const long long first = p.row0 + p.begin;
    const size_t seg = (size_t)k.slot * a.D;
    auto rows_of = [&](int i) { return i < tiles ? min(kTile, p.len - (tiles - 1 - i) * kTile) : 0; };
    if (threadIdx.x < kThreads) {  // the walk
        if (!ENDS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWalkRegs));
        const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, part = tid % S::L, n0 = 4 * part;
        const int c[2] = {tid / S::L, tid / S::L + S::HC}, turn = turn_of<NP>(tid);
        uint64_t A2[2][4];
        float carry[2][4], slowest[2];
        float2 dA[2][4] = {};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bool in = c[j] < k.channels;
            const size_t ch = (size_t)k.c0 + c[j];
            const Four Aj = scaled(load_states(a.A, ch, n0, a.N, in, turn), kLog2e);
            slowest[j] = slowest_of(Aj, n0, in ? a.N : 0, turn);
            Four g = {both(0.f), both(0.f)};
            if (!ENDS && p.len >= 0 && in) {  // from the segments behind this one
                const bool given = a.d_final && in_bounds(a.dbg, (size_t)p.seq, (size_t)a.tok.num_seqs, DBG_LOAD);
                g = load_states(a.d_final, (size_t)p.seq * a.D + ch, n0, a.N, given, turn);
                const int behind = (p.total + a.segment - 1) / a.segment - 1 - p.index;
                for (int i = k.slot + behind; i > k.slot; --i) {
                    const size_t at = (size_t)i * a.D + ch;
                    if (!in_bounds(a.dbg, at * NP + NP - 1, a.segment_floats, DBG_LOAD) ||
                        !in_bounds(a.dbg, at, a.sum_floats, DBG_LOAD))
                        break;
                    g = fma(decay(both(a.sums[at]), Aj, 0.f), g, four(*(const float4 *)(a.ends + at * NP + n0)));
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                A2[j][n] = twice(Aj.get(n));
                carry[j][n] = g.get(n);
            }
        }
        const long long tile0 = k.tiles0(a) + p.begin / kTile;
        auto states = [&](int i) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const size_t at = ((size_t)(2 * (tile0 + tiles - 1 - i) + half) * a.D + k.c0 + c[j]) * NP + n0;
                    const bool in = half * kHalf < rows_of(i) && c[j] < k.channels &&
                                    in_bounds(a.dbg, at + 3, a.saved_floats, DBG_LOAD);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     (uint32_t)__cvta_generic_to_shared(&s.h[ENDS ? 0 : i & 1][half][j][tid])),
                                 "l"(a.saved + (in ? at : 0)), "r"(in ? 16 : 0)
                                 : "memory");
                }
            cp_async_commit();
        };
        Phase phase(smem);
        if (!ENDS && tiles > 0) states(0);
        if (tiles > 0) sync_all();
        for (int i = 0; i < tiles; ++i) {
            const int b = i & 1;
            if (!ENDS) {
                states(i + 1);
                cp_async_wait_newest<1>();
            }
            phase.next();
            auto off = [&](const void *at) { return (uint32_t)((const char *)at - smem); };
            const uint32_t od[2] = {off(s.d[b] + place(c[0], 0)), off(s.d[b] + place(c[1], 0))};
            const uint32_t ox = off(s.x[b]) - off(s.d[b]), og = off(s.g[b]) - off(s.d[b]);
            uint32_t oB[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) oB[n] = off(&s.B[b][part][(n ^ turn) * kTile]);
            constexpr uint32_t toC = offsetof(M, C) - offsetof(M, B);
            const uint64_t raise = ENDS ? 0 : twice(raise_of(fminf(fabsf(phase.load(od[0])) * slowest[0],
                                                                   fabsf(phase.load(od[1])) * slowest[1])));
            // token t of a channel is at its place: groups of four change places (a XOR)
            auto at4 = [&](int j, int g) { return od[j] ^ (uint32_t)g << 4; };
            if (ENDS) {
#pragma unroll
                for (int g = kTile / 4 - 1; g >= 0; --g)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float2 d[2], gg[2];
                        phase.load4(at4(j, g), d);
                        phase.load4(at4(j, g) + og, gg);
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            float2 C[2];
                            phase.load4(oB[n] + toC + 16 * g, C);
#pragma unroll
                            for (int t = 1; t >= 0; --t) {
                                const float2 e = exponent(d[t], A2[j][n]), in = mul2(gg[t], C[t]);
                                carry[j][n] = (carry[j][n] + in.y) * ex2(e.y);
                                carry[j][n] = (carry[j][n] + in.x) * ex2(e.x);
                            }
                        }
                    }
            } else {
#pragma unroll 1
                for (int half = rows_of(i) > kHalf ? 1 : 0; half >= 0; --half) {
                    float h[2][4];
                    float2 P[2][4][4];  // p of a channel's state, of the half's pairs of tokens
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 v = s.h[ENDS ? 0 : b][half][j][tid];
                        h[j][0] = v.x; h[j][1] = v.y; h[j][2] = v.z; h[j][3] = v.w;
                    }
#pragma unroll
                    for (int gl = 0; gl < 2; ++gl) {
                        const int g = 2 * half + gl;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float2 d[2], x[2];
                            phase.load4(at4(j, g), d);
                            phase.load4(at4(j, g) + ox, x);
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                float2 B[2];
                                phase.load4(oB[n] + 16 * g, B);
#pragma unroll
                                for (int t = 0; t < 2; ++t) {
                                    const float2 e = fma2(d[t], A2[j][n], raise);
                                    float2 &pp = P[j][n][2 * gl + t];
                                    pp.x = ex2(e.x) * h[j][n];
                                    pp.y = ex2(e.y) * fmaf(x[t].x, B[t].x, pp.x);
                                    h[j][n] = fmaf(x[t].y, B[t].y, pp.y);
                                }
                            }
                        }
                    }
                    // back through the half, a pair of tokens at a time
#pragma unroll
                    for (int pi = 3; pi >= 0; --pi) {
                        const int g = 2 * half + pi / 2, t0 = half * kHalf + 2 * pi;
                        const uint32_t to = (pi & 1) * 8;
                        float2 B[4], C[4], dB[4], dC[4];
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            B[n] = phase.load2(oB[n] + 4 * t0);
                            C[n] = phase.load2(oB[n] + toC + 4 * t0);
                        }
                        using W = Share<S::L>;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t at = at4(j, g) + to;
                            const float2 d = phase.load2(at), x = phase.load2(at + ox), gg = phase.load2(at + og);
                            float2 s1, s2;
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                const float2 pp = P[j][n][pi];
                                const float2 e = fma2(d, A2[j][n], raise), hh = fma2(x, B[n], pp);
                                float2 G;
                                G.y = fmaf(gg.y, C[n].y, carry[j][n]);
                                G.x = fmaf(gg.x, C[n].x, G.y * ex2(e.y));
                                carry[j][n] = G.x * ex2(e.x);
                                const float2 gp = mul2(G, pp);
                                s1 = n ? fma2(G, B[n], s1) : mul2(G, B[n]);
                                s2 = n ? fma2(gp, A2[j][n], s2) : mul2(gp, A2[j][n]);
                                dA[j][n] = fma2(gp, d, dA[j][n]);
                                dB[n] = j ? fma2(G, x, dB[n]) : mul2(G, x);
                                dC[n] = j ? fma2(hh, gg, dC[n]) : mul2(hh, gg);
                            }
                            float v[4] = {s1.x, s1.y, s2.x, s2.y};
                            scatter_sum<S::L, 1>(v, tid);
                            if (W::mine(part)) {
#pragma unroll
                                for (int y = 0; y < W::kCount; ++y) {
                                    const int idx = W::first(part) + y;
                                    s.sum[ENDS ? 0 : b][idx >> 1][(t0 + (idx & 1)) * S::kRow + c[j]] = v[y];
                                }
                            }
                        }
                        constexpr int CW = 32 / S::L, kSame = CW > 8 ? CW / 8 : 1;
                        const int cl = lane / S::L;  // place among the warp's channels
#pragma unroll
                        for (int t = 1; t >= 0; --t) {
                            // half of the lanes go on with dB, half with dC; then a lane keeps the first
                            // of its numbers, which are other states in each
                            const bool up = cl & CW / 2;
                            float v[4];
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                const float x = t ? dB[n].y : dB[n].x, y = t ? dC[n].y : dC[n].x;
                                v[n] = (up ? y : x) + __shfl_xor_sync(0xffffffffu, up ? x : y, 16);
                            }
                            if (CW >= 4) {
#pragma unroll
                                for (int n = 0; n < 2; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n + 2], 8);
                            }
                            if (CW >= 8) v[0] += __shfl_xor_sync(0xffffffffu, v[1], 4);
                            if (CW >= 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
                            if (cl % kSame == 0) {
#pragma unroll
                                for (int n = 0; n < (CW >= 8 ? 1 : CW == 4 ? 2 : 4); ++n)
                                    s.bc[ENDS ? 0 : b][warp][t0 + t][(up ? NP : 0) + n0 + (n ^ turn)] = v[n];
                            }
                        }
                    }
                }
            }
            sync_all();
        }
        cp_async_wait_newest<0>();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const size_t ch = (size_t)k.c0 + c[j], at = (seg + ch) * NP + n0;
            if (c[j] >= k.channels) continue;
            const Four g = four(make_float4(carry[j][0], carry[j][1], carry[j][2], carry[j][3]));
            if (!ENDS && p.len >= 0 && p.begin == 0 && a.d_initial &&
                in_bounds(a.dbg, (size_t)p.seq, (size_t)a.tok.num_seqs, DBG_STORE))
                store_states(a.d_initial, (size_t)p.seq * a.D + ch, n0, a.N, g, turn);
            if (!in_bounds(a.dbg, at + 3, a.segment_floats, DBG_STORE)) continue;
            if (ENDS) {
                *(float4 *)(a.ends + at) = one(g);
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) a.part_A[at + (n ^ turn)] = dA[j][n].x + dA[j][n].y;
            }
        }
        return;
    }
    if (!ENDS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // this thread's chunks of a tile: tokens qt + x kStep, channels 8 q ..
    const int tid = threadIdx.x - kThreads;
    const int q = tid % S::kChunks, qt = tid / S::kChunks, qc = k.c0 + 8 * q, left = k.channels - 8 * q;
    constexpr int kStep = kThreads / S::kChunks;
    for (int i = tid; i < S::CH; i += kThreads) {
        s.param[0][i] = a.delta_bias && i < k.channels ? a.delta_bias[k.c0 + i] : 0.f;
        s.param[1][i] = a.skip && i < k.channels ? a.skip[k.c0 + i] : 0.f;
    }
    sync_half();
    auto bias = [&](int e) { return *(const float2 *)&s.param[0][8 * q + 2 * e]; };
    float2 dskip[4] = {}, dbias[4] = {};  // (ENDS: dskip is the sum of the step sizes)
    auto row_of = [&](int i) { return first + (tiles - 1 - i) * kTile; };
    auto fine = [&](int i) {
        return i >= tiles || in_bounds(a.dbg, (size_t)(row_of(i) + rows_of(i) - 1), (size_t)a.tok.rows(), DBG_LOAD);
    };
    auto fetch = [&](int i) {
        const int rows = fine(i) ? rows_of(i) : 0;
        auto &raw = s.raw[i % kStages];
#pragma unroll
        for (int x = 0; x < S::kPer; ++x) {
            const int t = qt + x * kStep;
            const bool ok = t < kTile && t < rows;
            const long long row = ok ? row_of(i) + t : 0;
            if (!ENDS) fetch_chunk<T>(&raw[0][x][tid], a.u, (const T *)a.u + row * a.u_stride + qc, left, ok, unit);
            fetch_chunk<T>(&raw[1][x][tid], a.delta, (const T *)a.delta + row * a.delta_stride + qc, left, ok, unit);
            fetch_chunk<T>(&raw[2][x][tid], a.dy, (const T *)a.dy + row * a.dy_stride + qc, left, ok, unit);
            if (a.z) fetch_chunk<T>(&raw[3][x][tid], a.z, (const T *)a.z + row * a.z_stride + qc, left, ok, unit);
        }
        cp_async_commit();
    };
    Vectors<T, NP> vb, vc;
    auto vectors = [&](int i) {
        const int rows = fine(i) ? rows_of(i) : 0;
        const long long row = rows ? row_of(i) : 0;
        if (!ENDS) vb.load(tid, a.B, a.B_stride, row, rows, k.group, a.N);
        vc.load(tid, a.C, a.C_stride, row, rows, k.group, a.N);
    };
    auto prepare = [&](int i) {
        const int rows = rows_of(i), b = i & 1;
        auto &raw = s.raw[i % kStages];
#pragma unroll
        for (int x = 0; x < S::kPer; ++x) {
            const int t = qt + x * kStep;
            if (t >= kTile) continue;
            const Vec<T, 8> dl = raw[1][x][tid], dy = raw[2][x][tid];
            Vec<T, 8> u, z;
            if (!ENDS) u = raw[0][x][tid];
            if (a.z) z = raw[3][x][tid];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 d = add2(pair(dl, e), bias(e)), g = pair(dy, e);
                if (a.softplus) d = softplus(d);
                if (t >= rows) d = both(0.f);
                if (a.z) {
                    const float2 zz = pair(z, e);
                    g = mul2(g, mul2(zz, sigmoid2(zz)));
                }
                const int at = place(8 * q + 2 * e, t >> 2) + (t & 3);
                s.d[b][at] = d.x;
                s.d[b][at + kTile] = d.y;
                s.g[b][at] = g.x;
                s.g[b][at + kTile] = g.y;
                if (ENDS) {
                    dskip[e] = add2(dskip[e], d);
                } else {
                    const float2 v = mul2(d, pair(u, e));
                    s.x[b][at] = v.x;
                    s.x[b][at + kTile] = v.y;
                }
            }
        }
        if (!ENDS) vb.put(tid, s.B[b]);
        vc.put(tid, s.C[b]);
    };
    // What the gate multiplies, on its way a tile ahead of its use.
    float2 open[S::kPer][4];
    const bool quads = a.D / a.G % 4 == 0;
    auto ungated = [&](int i) {
        const int rows = fine(i) ? rows_of(i) : 0;
#pragma unroll
        for (int x = 0; x < S::kPer; ++x) {
            const int t = qt + x * kStep;
            if (ENDS || !a.z || t >= kTile || t >= rows) continue;
            const float *at = open_row(a, row_of(i) + t) + qc;
            const bool there = left <= 0 || in_bounds(a.dbg, (size_t)(at - a.open) + min(left, 8) - 1, a.open_floats, DBG_LOAD);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (there && quads) {
                    if (4 * h < left) v = *(const float4 *)(at + 4 * h);
                } else if (there) {
                    if (4 * h < left) v.x = at[4 * h];
                    if (4 * h + 1 < left) v.y = at[4 * h + 1];
                    if (4 * h + 2 < left) v.z = at[4 * h + 2];
                    if (4 * h + 3 < left) v.w = at[4 * h + 3];
                }
                open[x][2 * h] = make_float2(v.x, v.y);
                open[x][2 * h + 1] = make_float2(v.z, v.w);
            }
        }
    };
    // What a tile's sums make: the gradients of its tokens (its d, x and g are this thread's own).
    auto finish = [&](int i) {
        const int rows = fine(i) ? rows_of(i) : 0, b = i & 1;
        auto &raw = s.raw[i % kStages];
#pragma unroll
        for (int x = 0; x < S::kPer; ++x) {
            const int t = qt + x * kStep;
            if (t >= kTile || t >= rows) continue;
            const long long row = row_of(i) + t;
            if (!in_bounds(a.dbg, (size_t)row, (size_t)a.tok.rows(), DBG_STORE)) continue;
            const Vec<T, 8> u = raw[0][x][tid], dl = raw[1][x][tid], dy = raw[2][x][tid];
            Vec<T, 8> z, du, dd, dz;
            if (a.z) z = raw[3][x][tid];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int cc = 8 * q + 2 * e, at = place(cc, t >> 2) + (t & 3), sat = t * S::kRow + cc;
                const float2 gb = *(const float2 *)&s.sum[b][0][sat], gpa = *(const float2 *)&s.sum[b][1][sat];
                const float2 d = make_float2(s.d[b][at], s.d[b][at + kTile]), skip = *(const float2 *)&s.param[1][cc];
                const float2 g = make_float2(s.g[b][at], s.g[b][at + kTile]), uu = pair(u, e);
                put_pair(du, e, fma2(d, gb, mul2(skip, g)));
                float2 v = fma2(uu, gb, mul2(gpa, both(kLn2)));
                if (a.softplus) v = mul2(v, sigmoid2(add2(pair(dl, e), bias(e))));
                put_pair(dd, e, v);
                dbias[e] = add2(dbias[e], v);
                dskip[e] = fma2(g, uu, dskip[e]);
                if (a.z) {
                    const float2 zz = pair(z, e), sg = sigmoid2(zz);
                    const float2 slope = mul2(sg, fma2(zz, fma2(sg, both(-1.f), both(1.f)), both(1.f)));
                    put_pair(dz, e, mul2(mul2(pair(dy, e), open[x][e]), slope));
                }
            }
            store_chunk(a.du, a.du_stride, row, qc, left, du, unit);
            store_chunk(a.ddelta, a.ddelta_stride, row, qc, left, dd, unit);
            if (a.z) store_chunk(a.dz, a.dz_stride, row, qc, left, dz, unit);
        }
        for (int e = tid; e < kTile * 2 * NP; e += kThreads) {
            const int t = e / (2 * NP), x = e % (2 * NP);
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += s.bc[b][w][t][x];
            const size_t at = (((size_t)k.blk * a.tok.rows() + row_of(i) + t) * a.G + k.group) * 2 * NP + x;
            if (t < rows && in_bounds(a.dbg, at, a.part_bc_floats, DBG_STORE)) a.part_bc[at] = v;
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
    for (int i = 0; i < tiles; ++i) {
        if (!ENDS && i > 0) finish(i - 1);
        ungated(i);
        if (i + 1 < tiles) {
            cp_async_wait_newest<kStages - 3>();
            prepare(i + 1);
            vectors(i + 2);
        }
        fetch(i + kStages - 1);
        sync_all();
    }
    if (!ENDS && tiles > 0) finish(tiles - 1);
    // sums of the threads of a chunk's channels, which each have some tokens
    sync_half();
    auto &sum = s.sum[0];
    if (qt < kTile) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int at = qt * S::kRow + 8 * q + 2 * e;
            sum[0][at] = dskip[e].x;
            sum[0][at + 1] = dskip[e].y;
            sum[1][at] = dbias[e].x;
            sum[1][at + 1] = dbias[e].y;
        }
    }
    sync_half();
    if (tid < k.channels) {
        float x = 0.f, y = 0.f;
        for (int t = 0; t < min(kTile, kStep); ++t) {
            x += sum[0][t * S::kRow + tid];
            y += sum[1][t * S::kRow + tid];
        }
        const size_t at = ENDS ? seg + k.c0 + tid : 2 * seg + k.c0 + tid;
        if (ENDS) {
            if (in_bounds(a.dbg, at, a.sum_floats, DBG_STORE)) a.sums[at] = x;
        } else if (in_bounds(a.dbg, at + a.D, a.part_D_floats, DBG_STORE)) {
            a.part_D[at] = x;
            a.part_D[at + a.D] = y;
        }
    }
    cp_async_wait_newest<0>();
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
    for (int b = 0; b < nb; ++b)
        if (in_bounds(a.dbg, b * step + i, a.part_bc_floats, DBG_LOAD)) s += a.part_bc[b * step + i];
    const size_t at = ((size_t)row * a.G + group) * a.N + n;
    if (in_bounds(a.dbg, at, (size_t)a.tok.rows() * a.G * a.N, DBG_STORE)) ((T *)(x < np ? a.dB : a.dC))[at] = from_f32<T>(s);
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
        for (int j = 0; j < slots; ++j)
            if (in_bounds(a.dbg, (size_t)(j * states + i), a.segment_floats, DBG_LOAD)) s += a.part_A[j * states + i];
        if (in_bounds(a.dbg, (size_t)(i / np * a.N + n), (size_t)a.D * a.N, DBG_STORE)) a.dA[i / np * a.N + n] = s;
    } else if (i < states + 2 * a.D) {
        const int x = (int)(i - states);
#pragma unroll 4
        for (int j = 0; j < slots; ++j)
            if (in_bounds(a.dbg, (size_t)j * 2 * a.D + x, a.part_D_floats, DBG_LOAD)) s += a.part_D[(size_t)j * 2 * a.D + x];
        float *to = x < a.D ? a.dskip : a.ddelta_bias;
        const int c = x < a.D ? x : x - a.D;
        if (to && in_bounds(a.dbg, (size_t)c, (size_t)a.D, DBG_STORE)) to[c] = s;
    }
}

template <typename T, int NP, bool ENDS>
cudaError_t walk(const ScanArgs &a, int nb, int unit, cudaStream_t stream) {
    constexpr int kBytes = sizeof(Smem<T, NP, ENDS>);
    static_assert(kBytes <= 227 * 1024, "");
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    // (with fewer registers at launch than it hands out, the walking half would wait for ever)
    if (e == cudaSuccess && !ENDS && (dev >= kMaxDev || !done[dev])) {
        cudaFuncAttributes f;
        e = cudaFuncGetAttributes(&f, kda_scan_bwd_kernel<T, NP, ENDS>);
        if (e == cudaSuccess && f.numRegs < kLaunchRegs) e = cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess) e = smem_limit_once(kda_scan_bwd_kernel<T, NP, ENDS>, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    return launch_early(kda_scan_bwd_kernel<T, NP, ENDS>, (unsigned)(a.tok.pieces(a.segment) * nb * a.G),
                        2 * kThreads, kBytes, stream, a, nb, unit);
}
template <typename T, int NP> cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    const int per = a.D / a.G, nb = (per + Shape<NP>::CH - 1) / Shape<NP>::CH;
    const long long slots = a.tok.pieces(a.segment);
    Unit u(a);
    u.add(a.u, a.u_stride);
    u.add(a.delta, a.delta_stride);
    u.add(a.z, a.z_stride);
    u.add(a.dy, a.dy_stride);
    u.add(a.du, a.du_stride);
    u.add(a.ddelta, a.ddelta_stride);
    u.add(a.dz, a.dz_stride);
    cudaError_t e = a.ends ? walk<T, NP, true>(a, nb, u.unit, stream) : cudaSuccess;
    if (e == cudaSuccess) e = walk<T, NP, false>(a, nb, u.unit, stream);
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
