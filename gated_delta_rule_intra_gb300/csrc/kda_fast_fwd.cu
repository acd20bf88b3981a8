// Forward of the gated delta-rule recurrence for BF16 training (see kda_fast.cuh): one CTA
// walks one (sequence, value head), or half of its dv columns, in steps of 16 tokens.
//
// A step passes four kinds of warps, three steps in flight: four warps turn the raw inputs into
// operand planes, four take the scores M and P, four solve the steps' triangular systems in
// turn, and eight (or four) consumers with 16 dv columns of the state each take the products.
// The walk is a chain, R -> e -> n -> S', so what bounds it is the time of one step on one SM:
// 3.7 thousand cycles with eight consumers, 2.9 with four.  A consumer's own 58 products are 0.5
// of these; the rest is shared by the issue slots and the shared-memory pipe (52% and 57% taken) and
// the chain's latencies.  With nothing but the consumers a step would take half as long.
// B=8 T=4096 H=16: 453 us for 256 steps, B=2 T=1024 H=4: 89 us for 64; with gates too strong for
// the mild form 504 and 101.
#include <type_traits>

#include "kda_fast.cuh"
#include "kda_ops.h"

namespace kda {
namespace fast {
namespace {

using chunk::bar_arrive;
using chunk::bar_or;
using chunk::bar_sync;
using chunk::cp16z;
using chunk::ldsm4;
using chunk::ldsm4t;
using chunk::plane_off;
using chunk::Seq;
using tc::smem_u32;

constexpr int kStages = 3;         // prepared stages
constexpr int kRaw = kStages + 2;  // raw input stages: two ahead, and as far back as a stage lives

// Named barriers; PLANES, FULL, EMPTY + stage, SOLVE + solver.
enum { BAR_PREP = 1, BAR_SCORE = 2, BAR_PLANES = 3, BAR_FULL = 6, BAR_EMPTY = 9, BAR_SOLVE = 12 };

constexpr int kSolvers = 4;  // warps that take the steps' systems in turn
// Mild steps are tried after as many that would have been: a step that turns out not to be is
// prepared twice (the first of a walk is, to find the planes' powers of two).
constexpr int kCalm = 4;
// NW consumer warps of 16 dv columns each; a head takes 8 / NW CTAs.
template <int NW> using Roles = chunk::Roles<NW, 8, kSolvers>;

enum { MILD = 0, GENERAL, STRONG };  // how a step's scores are taken

struct __align__(128) Stage {
    Planes pl;
    char t2[kTall];  // T2, FP32 for TF32 products
    char p[kTile];   // P, FP16
    float g[C][kRowPad];  // cumulative gate, unless the step is mild
    int form;
};

struct __align__(128) Smem {
    Stage stage[kStages];
    RawStage raw[kRaw];
    uint16_t v[kRaw][C][D];  // rows of the CTA's dv slice, swizzled chunks
    float beta[kRaw][C];
    float4 part[2][4][4][32];      // scores of a quarter of the channels, two steps' worth
    float a2[kSolvers][C][C + 4];  // (M diag(beta))^T
    float a1[kSolvers][C][C + 4];  // (diag(beta) M)^T
    char pt[kSolvers][kTall];      // P^T on its way to the saved tiles
    alignas(16) int mild[4];       // whether a preparing warp's part of a step would do for mild
    int big[kSolvers][4];          // whether a warp's entries of P are out of FP16's reach
    char out[8][512];          // a consumer's o on its way out
};

// A preparing thread's pointers to the raw inputs; step s is `s` steps further on.
template <int SLICE> struct Loader {
    const char *q, *v, *gate, *beta;  // (k lies as far from its start as q)
    long long row0;
    unsigned hrow, vrow;  // bytes of a token's row of q or k, and of v (gate: twice)
    int row, c, len;

    __device__ __forceinline__ Loader(const ChunkFwdArgs &a, const Seq &sq, int h, int hv, int dv0,
                                      int tid)
        : row0(sq.row0), row(tid >> 4), c(tid & 15), len(sq.len) {
        hrow = (unsigned)a.H * D * 2;
        vrow = (unsigned)a.HV * D * 2;
        const size_t r0 = (size_t)sq.row0;
        q = (const char *)a.q + r0 * hrow + h * D * 2 + c * 16;
        v = (const char *)a.v + r0 * vrow + (hv * D + dv0) * 2 + c * 16;
        gate = (const char *)a.gate + r0 * vrow * 2 + hv * D * 4 + c * 16;
        beta = (const char *)(a.beta + r0 * a.HV + hv);
    }
    __device__ __forceinline__ void load(Smem &sm, const ChunkFwdArgs &a, int step) const {
        const int slot = step % kRaw;
        RawStage &raw = sm.raw[slot];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = row + 8 * i, t = step * C + r;
            const bool ok = t < len && chunk::token_ok(a, row0 + t);
            const size_t at = ok ? (size_t)t : 0;
            cp16z(smem_u32(&raw.q[r][c * 8]), q + at * hrow, ok);
            cp16z(smem_u32(&raw.k[r][c * 8]), q + ((const char *)a.k - (const char *)a.q) + at * hrow, ok);
            cp16z(smem_u32(&raw.gate[r][c * 4]), gate + at * vrow * 2, ok);
            cp16z(smem_u32(&raw.gate[r][64 + c * 4]), gate + at * vrow * 2 + 256, ok);
            if (c < SLICE / 8)
                cp16z(smem_u32(sm.v[slot]) + plane_off(r, c), v + at * vrow, ok);
            if (c == 0)
                chunk::cp4z(smem_u32(&sm.beta[slot][r]), beta + at * a.HV * 4, ok);
        }
    }
};

// P's power of two: no entry is above 128 times the planes' largest elements, 2^13 with this.
__device__ __forceinline__ float p_scale(const Planes &p) {
    return 4.f * inverse_of(p.kinv * p.qinv);
}

// An entry of P (zero above the diagonal), `f` times as large in FP16.
__device__ __forceinline__ void put_p(Stage &out, char *pt, int r, int s, float x, float f) {
    const uint32_t b = pack_f16(x * f, 0.f);
    reinterpret_cast<uint16_t *>(out.p)[r * C + s] = (uint16_t)b;
    *reinterpret_cast<uint32_t *>(pt + tall_at(s, r)) = to_tf32(x);
}

// A warp's tile of the scores: M (w < 2) or P, the tokens s 8 (w % 2) on.  Entries above the
// diagonal may be of any size and are dropped.  Returns whether an entry of P is out of FP16's
// reach.
__device__ __forceinline__ bool put_scores(Smem &sm, Stage &out, const float *beta, int buf,
                                           const float (&x)[4], int w, int lane) {
    const int g = lane >> 2, t = lane & 3;
    bool big = false;
    const float f = p_scale(out.pl);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = g + (i >> 1) * 8, s = 8 * (w & 1) + 2 * t + (i & 1);
        if (w >= 2) {
            const float p = s <= r ? x[i] : 0.f;
            put_p(out, sm.pt[buf], r, s, p, f);
            big = big || !(fabsf(p) * f <= 16384.f);
        } else if (s < r) {
            sm.a2[buf][s][r] = x[i] * beta[s];
            sm.a1[buf][s][r] = x[i] * beta[r];
        }
    }
    return big;
}

// M and P of a mild step, M = kw (k 2^-g)^T and P = qw (k 2^-g)^T, from its planes.
__device__ __forceinline__ bool scores_mild(Smem &sm, Stage &out, const float *beta, int buf,
                                            int w, int lane) {
    const uint32_t left = smem_u32(w >= 2 ? out.pl.qw : out.pl.kw), right = smem_u32(out.pl.kd);
    const int m = lane >> 3, arow = (lane & 7) + (m & 1) * 8, brow = 8 * (w & 1) + (lane & 7);
    float c[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < 8; kk += 2) {
        uint32_t a0[4], a1[4], b[4];
        ldsm4(a0, left + plane_off(arow, 2 * kk + (m >> 1)));
        ldsm4(a1, left + plane_off(arow, 2 * kk + 2 + (m >> 1)));
        ldsm4(b, right + plane_off(brow, 2 * kk + m));
        mma_f16(c[0], a0, b[0], b[1]);
        mma_f16(c[1], a1, b[2], b[3]);
    }
    const float back =
        out.pl.kinv * (w >= 2 ? out.pl.qinv : out.pl.kinv) * (1.f / (1 << (kUp - kMildDown)));
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (c[0][i] + c[1][i]) * back;
    return put_scores(sm, out, beta, buf, x, w, lane);
}

// The same in general, in TF32: the exponents cancel in each term, and no term is above
// |q_r k_s|.  Each warp sums a quarter of the channels, straight from the raw inputs, then one of
// the four tiles over the quarters.
__device__ __forceinline__ bool scores(Smem &sm, Stage &out, const RawStage &raw,
                                       const float *beta, int buf, float scale, int w, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float acc[4][4] = {};  // M, tokens s 0-7 and 8-15; P, the same
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ch = 32 * w + 8 * i + 2 * t;
        uint32_t ak[4], aq[4], b[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = g + 8 * x;
            const float2 k = bf2(*reinterpret_cast<const uint32_t *>(&raw.k[r][ch]));
            const float2 q = bf2(*reinterpret_cast<const uint32_t *>(&raw.q[r][ch]));
            const float2 gg = *reinterpret_cast<const float2 *>(&out.g[r][ch]);
            const float2 up = make_float2(ex2(gg.x), ex2(gg.y));
            ak[x] = to_tf32(k.x * up.x);
            ak[2 + x] = to_tf32(k.y * up.y);
            aq[x] = to_tf32(scale * q.x * up.x);
            aq[2 + x] = to_tf32(scale * q.y * up.y);
            b[2 * x] = to_tf32(k.x * ex2(-gg.x));
            b[2 * x + 1] = to_tf32(k.y * ex2(-gg.y));
        }
        mma_tf32(acc[0], ak, b[0], b[1]);
        mma_tf32(acc[1], ak, b[2], b[3]);
        mma_tf32(acc[2], aq, b[0], b[1]);
        mma_tf32(acc[3], aq, b[2], b[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sm.part[buf & 1][w][i][lane] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    bar_sync(BAR_SCORE, kHalf);
    float x[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 y = sm.part[buf & 1][i][w][lane];
        x[0] += y.x; x[1] += y.y; x[2] += y.z; x[3] += y.w;
    }
    return put_scores(sm, out, beta, buf, x, w, lane);
}

// The same where 2^-g would leave FP32's range: pair by pair, one exp2 per (r, s, channel),
// every exponent <= 0.  17 pairs of the rows w and 15 - w a call; lane l holds channels 4l on.
__device__ __forceinline__ bool scores_strong(Smem &sm, Stage &out, const RawStage &raw,
                                              const float *beta, int buf, float scale, int w,
                                              int lane) {
    auto row4 = [&](const uint16_t *p, float (&x)[4]) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p + 4 * lane);
        const float2 lo = bf2(u.x), hi = bf2(u.y);
        x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
    };
    bool big = false;
    const float f = p_scale(out.pl);
#pragma unroll 1
    for (int j = 0; j < 17; ++j) {
        const int r = j <= w ? w : C - 1 - w, s = j <= w ? j : j - w - 1;
        float q[4], k[4], ks[4];
        row4(raw.q[r], q);
        row4(raw.k[r], k);
        row4(raw.k[s], ks);
        const float4 gr = *reinterpret_cast<const float4 *>(&out.g[r][4 * lane]);
        const float4 gs = *reinterpret_cast<const float4 *>(&out.g[s][4 * lane]);
        const float e[4] = {ex2(gr.x - gs.x) * ks[0], ex2(gr.y - gs.y) * ks[1],
                            ex2(gr.z - gs.z) * ks[2], ex2(gr.w - gs.w) * ks[3]};
        float p = 0.f, m = 0.f;
        for (int i = 0; i < 4; ++i) {
            p += q[i] * e[i];
            m += k[i] * e[i];
        }
        for (int off = 16; off > 0; off >>= 1) {
            p += __shfl_xor_sync(0xffffffffu, p, off);
            m += __shfl_xor_sync(0xffffffffu, m, off);
        }
        p *= scale;
        big = big || !(fabsf(p) * f <= 16384.f);
        if (lane == 0) {
            put_p(out, sm.pt[buf], r, s, p, f);
            if (s < r) {
                put_p(out, sm.pt[buf], s, r, 0.f, f);
                sm.a2[buf][s][r] = m * beta[s];
                sm.a1[buf][s][r] = m * beta[r];
            }
        }
    }
    return big;
}

// T2 = (I + M diag(beta))^-1 (lanes 0-15, one column each) and T = (I + diag(beta) M)^-1
// (lanes 16-31) by forward substitution in FP32, column by column of the matrix: a found entry
// is taken out of all later rows at once.  T goes to `tiles` as rows of T^T.
__device__ __forceinline__ void solve(Smem &sm, Stage &out, int buf, char *tiles, int lane) {
    const int c = lane & 15;
    const bool second = lane >= 16;
    const float(*A)[C + 4] = second ? sm.a1[buf] : sm.a2[buf];  // A[j][r], r > j
    float x[C];
#pragma unroll
    for (int r = 0; r < C; ++r) x[r] = r == c ? 1.f : 0.f;
#pragma unroll
    for (int j = 0; j < C - 1; ++j)
#pragma unroll
        for (int r = (j + 1) & ~3; r < C; r += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(&A[j][r]);
            if (r > j) x[r] -= a.x * x[j];
            if (r + 1 > j) x[r + 1] -= a.y * x[j];
            if (r + 2 > j) x[r + 2] -= a.z * x[j];
            x[r + 3] -= a.w * x[j];
        }
    if (!second) {
#pragma unroll
        for (int r = 0; r < C; ++r)
            *reinterpret_cast<uint32_t *>(out.t2 + tall_at(r, c)) = to_tf32(x[r]);
    } else if (tiles) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = (i >> 1) * 8 + (i & 1);
            *reinterpret_cast<uint4 *>(tiles + tall_off(c, i)) = make_uint4(
                to_tf32(x[b]), to_tf32(x[b + 2]), to_tf32(x[b + 4]), to_tf32(x[b + 6]));
        }
    }
}

template <int NW, bool SAVE>
__global__ void __launch_bounds__(Roles<NW>::kThreads, 1)
    kda_fast_fwd_kernel(const ChunkFwdArgs a) {
    wait_for_previous();
    constexpr int kSlice = 16 * NW, kSplit = D / kSlice;
    extern __shared__ __align__(128) char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int lane = threadIdx.x & 31;
    const Roles<NW> role(chunk::warp_index());
    const int unit = blockIdx.x / kSplit, dv0 = (blockIdx.x % kSplit) * kSlice;
    const int n = chunk::by_length(unit / a.HV, a.num_seqs, a.T, a.cu_seqlens);
    const int hv = unit - unit / a.HV * a.HV, h = hv / (a.HV / a.H);
    const Seq sq = chunk::seq_of(n, a.T, a.cu_seqlens);
    // whole 64-token slots where the backward's buffers are written: rows past the end are
    // computed as zeros, so every row of a slot is defined
    const int steps = SAVE ? (sq.len + BT - 1) / BT * (BT / C) : (sq.len + C - 1) / C;

    if (role.feeds) {
        role.give();
        if (role.prep >= 0) {
            const int tid = role.prep * 32 + lane;
            if (tid < kHalf) {  // raw inputs -> operand planes
                const Loader<kSlice> in(a, sq, h, hv, dv0, tid);
                for (int i = 0; i < 2; ++i) {
                    if (i < steps) in.load(sm, a, i);
                    cp_async_commit();
                }
                int calm = kCalm;  // steps in a row that were mild
                Scales sc;
                bool again = false;  // a step a second time, as the planes' powers did not fit
                for (int i = 0; i < steps;) {
                    const int st = i % kStages;
                    Stage &out = sm.stage[st];
                    cp_async_wait_newest<1>();
                    // the consumers are done with this stage's previous step (and its inputs)
                    if (i >= kStages && !again) bar_sync(BAR_EMPTY + st, kHalf + 32 * NW);
                    const RawStage &raw = sm.raw[i % kRaw];
                    bar_sync(BAR_PREP, kHalf);
                    int form = GENERAL;
                    if (calm >= kCalm && !again &&
                        !bar_or(BAR_PREP, kHalf, !prepare_mild(raw, out.pl, sc, a.scale, tid))) {
                        form = MILD;
                    } else {
                        const Seen f =
                            prepare<true, kUp, 0>(raw, out.pl, out.g, sc, a.scale, tid);
                        const bool mild = __all_sync(0xffffffffu, f.mild && f.in_range);
                        if (lane == 0) sm.mild[role.prep] = mild;
                        if (bar_or(BAR_PREP, kHalf, f.strong)) form = STRONG;
                        const bool off = bar_or(BAR_PREP, kHalf, !f.in_range);
                        const int4 m = *reinterpret_cast<const int4 *>(sm.mild);
                        calm = m.x && m.y && m.z && m.w ? calm + 1 : 0;
                        again = off && !again && !sc.fit(out.pl, a.scale);
                        if (again) {
                            sc.follow(out.pl, a.scale);
                            continue;
                        }
                    }
                    if (tid == 0) {
                        sc.put(out.pl);
                        out.form = form;
                    }
                    bar_arrive(BAR_PLANES + st, 2 * kHalf);
                    if (i + 2 < steps) in.load(sm, a, i + 2);
                    cp_async_commit();
                    ++i;
                }
                cp_async_wait_all();
                return;
            }
            // planes -> scores
            const int w = role.prep - kHalf / 32;
            for (int i = 0; i < steps; ++i) {
                const int st = i % kStages;
                Stage &out = sm.stage[st];
                const int buf = i % kSolvers;
                const float *beta = sm.beta[i % kRaw];
                const RawStage &raw = sm.raw[i % kRaw];
                bar_sync(BAR_PLANES + st, 2 * kHalf);
                bool big;
                const int form = chunk::uniform(out.form);
                if (form == MILD) {
                    big = scores_mild(sm, out, beta, buf, w, lane);
                } else if (form == GENERAL) {
                    big = scores(sm, out, raw, beta, buf, a.scale, w, lane);
                } else {
                    big = scores_strong(sm, out, raw, beta, buf, a.scale, w, lane);
                    big = scores_strong(sm, out, raw, beta, buf, a.scale, w + 4, lane) || big;
                }
                big = __any_sync(0xffffffffu, big);
                if (lane == 0) sm.big[buf][w] = big;
                bar_arrive(BAR_SOLVE + buf, kHalf + 32);
            }
            return;
        }
        if (role.solver >= 0) {  // scores -> T2 and T
            const int w = role.solver;
            for (int i = w; i < steps; i += kSolvers) {
                const int st = i % kStages;
                Stage &out = sm.stage[st];
                const float *beta = sm.beta[i % kRaw];
                char *tiles = nullptr;
                const size_t unit_at = (size_t)(sq.slot0 + i / 4) * a.HV + hv;
                if (SAVE && dv0 == 0 && dbg_ok(a.dbg, unit_at, a.units, DBG_STORE))
                    tiles = a.tiles + unit_at * kTilesBytes + (i % 4) * 2 * kTall;
                bar_sync(BAR_SOLVE + w, kHalf + 32);
                const uint4 *p = reinterpret_cast<const uint4 *>(sm.pt[w]);
                const uint4 p0 = p[lane], p1 = p[32 + lane];
                const float bm = warp_max(lane < C ? fabsf(beta[lane]) : 0.f);
                if (lane == 0) {
                    const int *big = sm.big[w];
                    out.pl.bmax = bm;
                    out.pl.careful = big[0] || big[1] || big[2] || big[3] || !finite(bm) ||
                                     !in_reach(out.pl, a.scale);
                }
                if (SAVE || lane < 16) solve(sm, out, w, tiles, lane);
                __syncwarp();
                bar_arrive(BAR_FULL + st, 32 + 32 * NW);
                if (tiles) {
                    uint4 *to = reinterpret_cast<uint4 *>(tiles + kTall);
                    to[lane] = p0;
                    to[32 + lane] = p1;
                }
            }
            return;
        }
        return;
    }

    // ------------------------------------------------------------------ consumers
    role.take();
    if (role.consumer < 0) return;
    const int tile0 = dv0 / 16 + role.consumer;  // the head's tile of 16 dv columns
    const int tc2 = (lane & 3) * 2;
    const int lrow = (lane & 7) + ((lane >> 4) & 1) * 8, lcol = (lane >> 3) & 1;
    const int trow = lane & 15, tcol = lane >> 4;
    Tile S;
    S.clear();
    const size_t orow = (size_t)a.HV * D;
    uint16_t *o_at = (uint16_t *)a.o + (size_t)sq.row0 * orow + (size_t)hv * D + tile0 * 16;

    for (int i = 0; i < steps; ++i) {
        const int st = i % kStages, slot = i % kRaw;
        const unsigned unit_at = (unsigned)(sq.slot0 + i / 4) * a.HV + hv;
        bar_sync(BAR_FULL + st, 32 + 32 * NW);
        const Stage &in = sm.stage[st];
        const float *beta = sm.beta[slot];
        const uint32_t kw = smem_u32(in.pl.kw), qw = smem_u32(in.pl.qw), kd = smem_u32(in.pl.kd);
        const float kinv = in.pl.kinv, qinv = in.pl.qinv, ktop = largest(in.pl.kmax);
        const bool save = SAVE && dbg_ok(a.dbg, unit_at, a.units, DBG_STORE);
        const bool keep = save && i % 4 == 0;
        bool careful = chunk::uniform(in.pl.careful);
        if (chunk::uniform(S.bound > kLimit)) S.renew();
        uint32_t th[4], tl[4], pf[4];
        load_tall(smem_u32(in.t2), lane, tl, th);
        ldsm4(pf, smem_u32(in.p) + chunk::tile_lane(lane));
        const float2 b[2] = {*reinterpret_cast<const float2 *>(&beta[tc2]),
                             *reinterpret_cast<const float2 *>(&beta[8 + tc2])};
        float xw[2][4] = {}, xq[2][4] = {}, e[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            uint32_t kf[4], qf[4];
            const uint32_t off = plane_off(lrow, 2 * kk + lcol);
            ldsm4(kf, kw + off);
            ldsm4(qf, qw + off);
            const float(&x)[4] = S.s[2 * kk], (&y)[4] = S.s[2 * kk + 1];
            const uint32_t af[4] = {pack_f16(x[0], x[1]), pack_f16(x[2], x[3]),
                                    pack_f16(y[0], y[1]), pack_f16(y[2], y[3])};
            mma_f16(xw[0], af, kf[0], kf[1]);
            mma_f16(xw[1], af, kf[2], kf[3]);
            mma_f16(xq[0], af, qf[0], qf[1]);
            mma_f16(xq[1], af, qf[2], qf[3]);
        }
        if (keep)  // outside the loop above, which a branch would cut into pieces
            store_tile(a.ckpt + unit_at * kCkptBytes, S, tile0, lane);
        const bool mild = chunk::uniform(in.form == MILD);
        const float ckpt_scale = S.saved_scale();  // of the state as an operand
        const float inv = S.inv * (1.f / (1 << kUp));
        // R = v - kw S and e = T2 R; blocks (tokens 0-7, dv 0-7), (0-7, 8-15), (8-15, ..)
        uint32_t vr[4], x0[4], x1[4];
        ldsm4t(vr, smem_u32(sm.v[slot]) + plane_off(lrow, role.consumer * 2 + lcol));
        float R[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 x = bf2(vr[2 * j]), y = bf2(vr[2 * j + 1]);
            const float back = -inv * kinv;
            R[j][0] = fmaf(xw[j][0], back, x.x);
            R[j][1] = fmaf(xw[j][1], back, x.y);
            R[j][2] = fmaf(xw[j][2], back, y.x);
            R[j][3] = fmaf(xw[j][3], back, y.y);
        }
        tf_frag(R[0], x0);
        tf_frag(R[1], x1);
        mma_tall(e[0], e[1], x0, x1, tl, th);
        float em = warp_max(abs_max(e));
        careful = careful || !finite(em);
        const float bm = in.pl.bmax;
        if (!chunk::uniform(careful)) {
            // n = beta e with the inverse of the key plane's power of two
            const float less = mild ? 1.f / (1 << kMildDown) : 1.f;
            const float more = (mild ? (float)(1 << kMildDown) : 1.f) * kinv;
            uint32_t nf[4];
            const float ratio = join_scale(S, em * bm * more, em * bm * (C * ktop));
            const float c = S.c * more;
            nf[0] = pack_f16(e[0][0] * (b[0].x * c), e[0][1] * (b[0].y * c));
            nf[1] = pack_f16(e[0][2] * (b[0].x * c), e[0][3] * (b[0].y * c));
            nf[2] = pack_f16(e[1][0] * (b[1].x * c), e[1][1] * (b[1].y * c));
            nf[3] = pack_f16(e[1][2] * (b[1].x * c), e[1][3] * (b[1].y * c));
            S.inv = inverse_of(S.c);
            // S' = diag(2^g_l) (S + (k 2^-g)^T n), or diag(2^g_l) S + kd^T n
            if (mild && chunk::uniform(ratio != 1.f)) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
#pragma unroll
                    for (int p = 0; p < 4; ++p) S.s[j][p] *= ratio;
            }
            auto update = [&](auto decay_last) {
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
                    uint32_t kf[4];
                    ldsm4t(kf, kd + plane_off(trow, 2 * jj + tcol));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float2 d =
                            *reinterpret_cast<const float2 *>(&in.pl.decay[16 * jj + 8 * x + tc2]);
                        float(&s)[4] = S.s[2 * jj + x];
                        const float2 dr =
                            decay_last ? d : chunk::mul2(d, make_float2(ratio, ratio));
                        if (decay_last) mma_f16(s, nf, kf[2 * x], kf[2 * x + 1]);
                        const float2 u = chunk::mul2(make_float2(s[0], s[1]), dr);
                        const float2 w = chunk::mul2(make_float2(s[2], s[3]), dr);
                        s[0] = u.x; s[1] = u.y; s[2] = w.x; s[3] = w.y;
                        if (!decay_last) mma_f16(s, nf, kf[2 * x], kf[2 * x + 1]);
                    }
                }
            };
            if (mild)
                update(std::true_type{});
            else
                update(std::false_type{});
            // o = qw S + P n
            float po[2][4] = {};
            mma_f16(po[0], nf, pf[0], pf[1]);
            mma_f16(po[1], nf, pf[2], pf[3]);
            const float p_inv = S.inv * less * (qinv / 4.f), q_inv = inv * qinv;  // see p_scale()
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int p = 0; p < 4; ++p) xq[j][p] = fmaf(po[j][p], p_inv, xq[j][p] * q_inv);
        } else {
            walk_tokens(S, xq, e, sm.raw[slot], beta, sm.v[slot], role.consumer * 16, a.scale,
                        lane);
            em = warp_max(abs_max(e));
        }
        if (i + kStages < steps) bar_arrive(BAR_EMPTY + st, kHalf + 32 * NW);
        if (save) {
            const float s =
                store_block(a.e + unit_at * kRowsBytes, e, em, (i % 4) * 8 + tile0, lane);
            if (lane == 0) {
                float *scales = a.scales + unit_at * kScales + tile0;
                scales[8 + (i % 4) * 8] = s;
                if (keep) scales[0] = ckpt_scale;
            }
        }
        uint32_t ow[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            ow[2 * j] = chunk::pack_bf16(xq[j][0], xq[j][1]);
            ow[2 * j + 1] = chunk::pack_bf16(xq[j][2], xq[j][3]);
        }
        chunk::store_out(sm.out[role.consumer], ow, (char *)(o_at + (size_t)i * C * orow),
                         orow * 2, sq.len - i * C, (char *)a.o, a.rows_o * D * 2, a.dbg, lane);
    }
}

template <int NW, bool SAVE>
cudaError_t launch(const ChunkFwdArgs &a, int dev, cudaStream_t stream) {
    static volatile int done[kMaxDev];
    cudaError_t e = chunk::ready_once<Roles<NW>>(kda_fast_fwd_kernel<NW, SAVE>,
                                            (int)sizeof(Smem), dev, done);
    if (e != cudaSuccess) return e;
    const int grid = a.num_seqs * a.HV * (8 / NW);
    return launch_early(kda_fast_fwd_kernel<NW, SAVE>, grid, Roles<NW>::kThreads, sizeof(Smem),
                        stream, a);
}

template <bool SAVE> cudaError_t launch_split(const ChunkFwdArgs &a, int dev, cudaStream_t stream) {
    // A step takes 3.7 thousand cycles in one CTA a head and 2.9 in two.  In four it takes
    // as long: the preparation bounds it from two on.
    return chunk::best_split(a.num_seqs, a.HV, a.cu_seqlens) == 1
               ? launch<8, SAVE>(a, dev, stream)
               : launch<4, SAVE>(a, dev, stream);
}

}  // namespace

cudaError_t launch_fwd(const ChunkFwdArgs &a, int dev, cudaStream_t stream) {
    return a.ckpt ? launch_split<true>(a, dev, stream) : launch_split<false>(a, dev, stream);
}

}  // namespace fast
}  // namespace kda
