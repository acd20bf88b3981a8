// Backward of the gated delta-rule recurrence for BF16 training, first pass (see kda_fast.cuh,
// and kda_chunk_bwd_state.cu for what it computes): the state's gradient walks each
// (sequence, value head) backwards in steps of 16 tokens.
//
// Bound as the forward is, by the time of a step on one SM: 3.1 thousand cycles with eight
// consumers (B=8 T=4096 H=16: 388 us), 2.2 with four, 1.8 with two (B=2 T=1024 H=4: 57 us).
// Nothing is solved here (T comes from the forward), so that two groups of four preparing warps,
// each with every second step, keep ahead of the consumers.
#include "kda_fast.cuh"
#include "kda_ops.h"

namespace kda {
namespace fast {
namespace {

using chunk::bar_arrive;
using chunk::bar_sync;
using chunk::cp16z;
using chunk::ldsm4;
using chunk::ldsm4t;
using chunk::plane_off;

template <int NW> using Roles = chunk::Roles<NW, 8, 0>;
using chunk::Seq;
using tc::smem_u32;

constexpr int kStages = 3, kRaw = kStages + 2;

enum { BAR_PREP = 1, BAR_FULL = 3, BAR_EMPTY = 6 };  // PREP + group; FULL, EMPTY + stage

struct __align__(128) Smem {
    Planes stage[kStages];
    RawStage raw[kRaw];
    uint16_t dout[kRaw][C][D];  // rows of the CTA's dv slice, swizzled chunks
    char tiles[kRaw][2 * kTall];
    float beta[kRaw][C];
    char out[8][512];  // a consumer's dv on its way out
};

// Step i of the walk (the last step of the sequence first), tokens 16 * step on.
template <int SLICE>
__device__ __forceinline__ void load_step(Smem &sm, const ChunkBwdArgs &a, const Seq &sq, int h,
                                          int hv, int dv0, int i, int step, int tid) {
    const int slot = i % kRaw, c = tid & 15;
    RawStage &raw = sm.raw[slot];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int r = (tid >> 4) + 8 * x, t = step * C + r;
        const bool ok = t < sq.len && chunk::token_ok(a, sq.row0 + t);
        const size_t tok = (size_t)sq.row0 + (ok ? t : 0);
        const size_t iq = (tok * a.H + h) * D + c * 8, iv = (tok * a.HV + hv) * D;
        cp16z(smem_u32(&raw.q[r][c * 8]), (const uint16_t *)a.q + iq, ok);
        cp16z(smem_u32(&raw.k[r][c * 8]), (const uint16_t *)a.k + iq, ok);
        cp16z(smem_u32(&raw.gate[r][c * 4]), a.gate + iv + c * 4, ok);
        cp16z(smem_u32(&raw.gate[r][64 + c * 4]), a.gate + iv + 64 + c * 4, ok);
        if (c < SLICE / 8)
            cp16z(smem_u32(sm.dout[slot]) + plane_off(r, c),
                  (const uint16_t *)a.dout + iv + dv0 + c * 8, ok);
        if (c == 0) chunk::cp4z(smem_u32(&sm.beta[slot][r]), a.beta + tok * a.HV + hv, ok);
    }
    const size_t unit_at = (size_t)(sq.slot0 + step / 4) * a.HV + hv;
    if (dbg_ok(a.dbg, unit_at, a.units, DBG_LOAD))
        cp16z(smem_u32(sm.tiles[slot]) + tid * 16,
              a.tiles + unit_at * kTilesBytes + (step % 4) * 2 * kTall + tid * 16, true);
}

template <int NW>
__global__ void __launch_bounds__(Roles<NW>::kThreads, 1)
    kda_fast_bwd_state_kernel(const ChunkBwdArgs a) {
    constexpr int kSlice = 16 * NW, kSplit = D / kSlice;
    extern __shared__ __align__(128) char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int lane = threadIdx.x & 31;
    const Roles<NW> role(chunk::warp_index());
    const int unit = blockIdx.x / kSplit, dv0 = (blockIdx.x % kSplit) * kSlice;
    const int n = chunk::by_length(unit / a.HV, a.num_seqs, a.T, a.cu_seqlens);
    const int hv = unit % a.HV, h = hv / (a.HV / a.H);
    const Seq sq = chunk::seq_of(n, a.T, a.cu_seqlens);
    const int steps = (sq.len + BT - 1) / BT * (BT / C);

    if (role.feeds) {
        role.give();
        if (role.prep >= 0) {
            // two groups of four warps take the steps in turn
            const int group = role.prep >> 2, tid = (role.prep & 3) * 32 + lane;
            if (group < steps)
                load_step<kSlice>(sm, a, sq, h, hv, dv0, group, steps - 1 - group, tid);
            cp_async_commit();
            for (int i = group; i < steps; i += 2) {
                const int st = i % kStages;
                Planes &out = sm.stage[st];
                // the consumers are done with this stage's previous step and its inputs, whose
                // place the step after next takes
                if (i >= kStages) bar_sync(BAR_EMPTY + st, kHalf + 32 * NW);
                if (i + 2 < steps)
                    load_step<kSlice>(sm, a, sq, h, hv, dv0, i + 2, steps - 3 - i, tid);
                cp_async_commit();
                cp_async_wait_newest<1>();
                find_largest(sm.raw[i % kRaw], out, tid);
                bar_sync(BAR_PREP + group, kHalf);
                Scales sc;
                sc.follow(out, a.scale);
                if (tid == 32) {
                    sc.put(out);
                    out.ktop = largest(out.kmax);
                    out.qtop = fabsf(a.scale) * largest(out.qmax);
                }
                // kw and qw are added to the state's gradient, kd is only multiplied by it
                prepare<false, 0, kUp>(sm.raw[i % kRaw], out, nullptr, sc, a.scale, tid);
                if (tid < 32) {
                    const float bm =
                        warp_max(lane < C ? fabsf(sm.beta[i % kRaw][lane]) : 0.f);
                    if (lane == 0) {
                        out.bmax = bm;
                        out.careful = !finite(bm) || !in_reach(out, a.scale);
                    }
                }
                bar_arrive(BAR_FULL + st, kHalf + 32 * NW);
            }
            cp_async_wait_all();
            return;
        }
        return;
    }

    role.take();
    if (role.consumer < 0) return;
    const int tile0 = dv0 / 16 + role.consumer;
    const int gr = lane >> 2, tc2 = (lane & 3) * 2;
    const int lrow = (lane & 7) + ((lane >> 4) & 1) * 8, lcol = (lane >> 3) & 1;
    const int trow = lane & 15, tcol = lane >> 4;
    Tile S;
    const size_t sbase = ((size_t)n * a.HV + hv) * D * D + (size_t)tc2 * D + tile0 * 16 + gr;
    S.clear();
    const bool states_in = chunk::state_ok(a, a.d_final_state, sbase, DBG_LOAD) &&
                           chunk::state_ok(a, a.d_initial_state, sbase, DBG_STORE);
    if (a.d_final_state && states_in) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float *p = a.d_final_state + sbase + (size_t)8 * j * D;
            S.s[j][0] = p[0];
            S.s[j][1] = p[D];
            S.s[j][2] = p[8];
            S.s[j][3] = p[D + 8];
        }
        S.bound = 2.f * kLimit;
    }
    const size_t vrow = (size_t)a.HV * D;
    uint16_t *dv_at = (uint16_t *)a.dv + (size_t)sq.row0 * vrow + (size_t)hv * D + tile0 * 16;

    for (int i = 0; i < steps; ++i) {
        const int st = i % kStages, slot = i % kRaw, step = steps - 1 - i;
        const unsigned unit_at = (unsigned)(sq.slot0 + step / 4) * a.HV + hv;
        const bool save = dbg_ok(a.dbg, unit_at, a.units, DBG_STORE), keep = save && step % 4 == 3;
        bar_sync(BAR_FULL + st, kHalf + 32 * NW);
        const Planes &in = sm.stage[st];
        const uint32_t kw = smem_u32(in.kw), qw = smem_u32(in.qw), kd = smem_u32(in.kd);
        const float kinv = in.kinv, qinv = in.qinv, ktop = in.ktop, qtop = in.qtop, bm = in.bmax;
        bool careful = in.careful;
        if (chunk::uniform(S.bound > kLimit)) S.renew();
        uint32_t th[4], tl[4], ph[4], pl[4];
        load_tall(smem_u32(sm.tiles[slot]), lane, tl, th);
        load_tall(smem_u32(sm.tiles[slot]) + kTall, lane, pl, ph);
        const float2 b[2] = {*reinterpret_cast<const float2 *>(&sm.beta[slot][tc2]),
                             *reinterpret_cast<const float2 *>(&sm.beta[slot][8 + tc2])};
        uint32_t dor[4];  // do^T, BF16 pairs of tokens
        float ds[2][4] = {};
        ldsm4t(dor, smem_u32(sm.dout[slot]) + plane_off(lrow, role.consumer * 2 + lcol));
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __vmaxu2(m, dor[j] & 0x7fff7fffu);
        const float om = __uint_as_float(
            __reduce_max_sync(0xffffffffu, max(m << 16, m & 0xffff0000u)));
        // dS' kd
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            uint32_t kf[4];
            ldsm4(kf, kd + plane_off(lrow, 2 * kk + lcol));
            const float(&x)[4] = S.s[2 * kk], (&y)[4] = S.s[2 * kk + 1];
            const uint32_t af[4] = {pack_f16(x[0], x[1]), pack_f16(x[2], x[3]),
                                    pack_f16(y[0], y[1]), pack_f16(y[2], y[3])};
            mma_f16(ds[0], af, kf[0], kf[1]);
            mma_f16(ds[1], af, kf[2], kf[3]);
        }
        if (keep)  // outside the loop above, which a branch would cut into pieces
            store_tile(a.dckpt + unit_at * kCkptBytes, S, tile0, lane);
        const float ckpt_scale = S.saved_scale();
        float y[2][4] = {};
        // dn^T = do^T P + dS'^T kd^T (do is exact in TF32), Y^T = dn^T T
        float dn[2][4] = {};
        const uint32_t o0[4] = {dor[0] << 16, dor[1] << 16, dor[0] & 0xffff0000u,
                                dor[1] & 0xffff0000u};
        const uint32_t o1[4] = {dor[2] << 16, dor[3] << 16, dor[2] & 0xffff0000u,
                                dor[3] & 0xffff0000u};
        mma_tall(dn[0], dn[1], o0, o1, pl, ph);
        uint32_t x0[4], x1[4];
        const float ds_inv = S.inv * (1.f / (1 << kUp)) * kinv;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p) dn[j][p] = fmaf(ds[j][p], ds_inv, dn[j][p]);
        tf_frag(dn[0], x0);
        tf_frag(dn[1], x1);
        mma_tall(y[0], y[1], x0, x1, tl, th);
        float ym = warp_max(abs_max(y));
        careful = careful || !finite(ym) || !finite(om);
        if (!chunk::uniform(careful)) {
            uint32_t of[4], nf[4];
            const float ratio = join_scale(S, fmaxf(om * qinv, ym * bm * kinv),
                                           C * (om * qtop + ym * bm * ktop));
            const float c = S.c, co = c * qinv, cy = c * kinv;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 o = bf2(dor[j]);
                of[j] = pack_f16(o.x * co, o.y * co);
            }
            const float nx[2] = {-b[0].x * cy, -b[1].x * cy}, ny[2] = {-b[0].y * cy, -b[1].y * cy};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                nf[2 * j] = pack_f16(y[j][0] * nx[j], y[j][1] * ny[j]);
                nf[2 * j + 1] = pack_f16(y[j][2] * nx[j], y[j][3] * ny[j]);
            }
            S.inv = inverse_of(c);
            // dS = diag(2^g_l) dS' + qw^T do - kw^T dv
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) {
                uint32_t kf[4], qf[4];
                ldsm4t(qf, qw + plane_off(trow, 2 * jj + tcol));
                ldsm4t(kf, kw + plane_off(trow, 2 * jj + tcol));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float2 d =
                        *reinterpret_cast<const float2 *>(&in.decay[16 * jj + 8 * x + tc2]);
                    float(&s)[4] = S.s[2 * jj + x];
                    const float2 dr = chunk::mul2(d, make_float2(ratio, ratio));
                    const float2 u = chunk::mul2(make_float2(s[0], s[1]), dr);
                    const float2 w = chunk::mul2(make_float2(s[2], s[3]), dr);
                    s[0] = u.x; s[1] = u.y; s[2] = w.x; s[3] = w.y;
                    mma_f16(s, of, qf[2 * x], qf[2 * x + 1]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    mma_f16(S.s[2 * jj + x], nf, kf[2 * x], kf[2 * x + 1]);
            }
        } else {
            walk_tokens_back(S, y, sm.raw[slot], sm.beta[slot], sm.dout[slot],
                             role.consumer * 16, a.scale, lane);
            ym = warp_max(abs_max(y));
        }
        if (i + kStages < steps) bar_arrive(BAR_EMPTY + st, kHalf + 32 * NW);
        uint32_t dw[4];  // dv = beta Y
        float s = 1.f;
        if (save) s = store_block(a.y + unit_at * kRowsBytes, y, ym, (step % 4) * 8 + tile0, lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            dw[2 * j] = chunk::pack_bf16(b[j].x * y[j][0], b[j].y * y[j][1]);
            dw[2 * j + 1] = chunk::pack_bf16(b[j].x * y[j][2], b[j].y * y[j][3]);
        }
        if (save && lane == 0) {
            float *scales = a.dscales + unit_at * kScales + tile0;
            scales[8 + (step % 4) * 8] = s;
            if (keep) scales[0] = ckpt_scale;
        }
        chunk::store_out(sm.out[role.consumer], dw, (char *)(dv_at + (size_t)step * C * vrow),
                         vrow * 2, sq.len - step * C, (char *)a.dv, a.rows_o * D * 2, a.dbg, lane);
    }
    if (a.d_initial_state && states_in) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float *p = a.d_initial_state + sbase + (size_t)8 * j * D;
            p[0] = S.s[j][0] * S.inv;
            p[D] = S.s[j][1] * S.inv;
            p[8] = S.s[j][2] * S.inv;
            p[D + 8] = S.s[j][3] * S.inv;
        }
    }
}

template <int NW>
cudaError_t launch(const ChunkBwdArgs &a, int dev, cudaStream_t stream) {
    static volatile int done[kMaxDev];
    cudaError_t e = chunk::ready_once<Roles<NW>>(kda_fast_bwd_state_kernel<NW>,
                                            (int)sizeof(Smem), dev, done);
    if (e != cudaSuccess) return e;
    kda_fast_bwd_state_kernel<NW><<<a.num_seqs * a.HV * (8 / NW), Roles<NW>::kThreads,
                                    sizeof(Smem), stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_state(const ChunkBwdArgs &a, int dev, cudaStream_t stream) {
    switch (chunk::best_split(a.num_seqs, a.HV, a.cu_seqlens)) {
        case 1: return launch<8>(a, dev, stream);
        case 2: return launch<4>(a, dev, stream);
        default: return launch<2>(a, dev, stream);
    }
}

}  // namespace fast
}  // namespace kda
