// Backward of the gated delta-rule recurrence, first pass: the state's gradient walks each
// (sequence, value head) backwards in steps of 16 tokens, as the forward walks it forwards
// (see kda_chunk.cuh).  Writes dv, Y (the gradient of beta e's source, dv = beta Y) and the
// state's gradient at the end of each 64-token slot, from which the second pass takes the
// other gradients of all slots at once.
//
// Bound by the time of a step on one SM, as the forward: B=8 T=2048 H=16 FP16 in one CTA a head
// 330 us for 128 steps (5.3 thousand cycles); 9 packed sequences of up to 4096 tokens, 8 value
// heads, in four CTAs a head 302 us for the longest's 256 (2.4).
#include <type_traits>

#include "kda_chunk.cuh"
#include "kda_ops.h"

namespace kda {
namespace chunk {
namespace {

constexpr int kRaw = 3, kRing = 4, kStages = 2;

// FULL, EMPTY + stage; JOIN + pair of consumers that share a tile
enum { BAR_PREP = 1, BAR_FULL = 2, BAR_EMPTY = 4, BAR_JOIN = 6 };

struct __align__(128) Prepared {
    char planes[kPlanes * kPlane];
    float decay[D];
};

struct __align__(128) Smem {
    Prepared prep[kStages];
    RawStage raw[kRaw];
    uint16_t dout[kRing][C][D];   // rows of the CTA's dv slice, swizzled chunks
    char tiles[kRing][kTilesBytes];
    float beta[kRing][C];
    float4 join[2][4][2][32];  // partial sums of consumers that share a tile, two steps' worth
};

// Step i of the walk (the last step of the sequence first): token 16 * step on.
template <int SLICE>
__device__ __forceinline__ void load_step(Smem &sm, const ChunkBwdArgs &a, const Seq &sq, int h,
                                          int hv, int dv0, int i, int step, int tid) {
    const int row = tid >> 4, c = tid & 15;
    const int t = step * C + row;
    const bool ok = t < sq.len && token_ok(a, sq.row0 + t);
    const size_t tok = (size_t)sq.row0 + (ok ? t : 0);
    RawStage &raw = sm.raw[i % kRaw];
    const size_t iq = (tok * a.H + h) * D + c * 8, iv = (tok * a.HV + hv) * D;
    cp16z(tc::smem_u32(&raw.q[row][c * 8]), (const uint16_t *)a.q + iq, ok);
    cp16z(tc::smem_u32(&raw.k[row][c * 8]), (const uint16_t *)a.k + iq, ok);
    cp16z(tc::smem_u32(&raw.gate[row][c * 4]), a.gate + iv + c * 4, ok);
    cp16z(tc::smem_u32(&raw.gate[row][64 + c * 4]), a.gate + iv + 64 + c * 4, ok);
    if (c < SLICE / 8)
        cp16z(tc::smem_u32(sm.dout[i % kRing]) + plane_off(row, c),
              (const uint16_t *)a.dout + iv + dv0 + c * 8, ok);
    if (c == 0) cp4z(tc::smem_u32(&sm.beta[i % kRing][row]), a.beta + tok * a.HV + hv, ok);
    const size_t unit_at = (size_t)(sq.slot0 + step / 4) * a.HV + hv;
    if (tid < (int)kTilesBytes / 16 && dbg_ok(a.dbg, unit_at, a.units, DBG_LOAD))
        cp16z(tc::smem_u32(sm.tiles[i % kRing]) + tid * 16,
              a.tiles + (unit_at * 4 + step % 4) * kTilesBytes + tid * 16, true);
}

// Four tiles += A B with A of the inputs: exact in BF16 (no lo part), split in two for FP16.
template <bool EXACT>
__device__ __forceinline__ void mma_in(float (&c0)[4], float (&c1)[4], float (&d0)[4],
                                       float (&d1)[4], const uint32_t (&ah)[4],
                                       const uint32_t (&al)[4], const uint32_t (&bh)[4],
                                       const uint32_t (&bl)[4], const uint32_t (&yh)[4],
                                       const uint32_t (&yl)[4]) {
    mma16816(c0, ah, bh[0], bh[1]);
    mma16816(c1, ah, bh[2], bh[3]);
    mma16816(d0, ah, yh[0], yh[1]);
    mma16816(d1, ah, yh[2], yh[3]);
    mma16816(c0, ah, bl[0], bl[1]);
    mma16816(c1, ah, bl[2], bl[3]);
    mma16816(d0, ah, yl[0], yl[1]);
    mma16816(d1, ah, yl[2], yl[3]);
    if (!EXACT) {
        mma16816(c0, al, bh[0], bh[1]);
        mma16816(c1, al, bh[2], bh[3]);
        mma16816(d0, al, yh[0], yh[1]);
        mma16816(d1, al, yh[2], yh[3]);
    }
}

// NC consumer warps, KS for each 16 dv columns: a head takes 8 KS / NC CTAs.  With KS = 2 a warp
// has half of dk: sums over dk are joined with the partner's in shared memory, both have Y, and
// each writes the Y and dv of its half of the tokens.
template <typename T16, int NC, int KS>
__global__ void __launch_bounds__(Roles<NC, 8, 0>::kThreads, 1)
    kda_chunk_bwd_state_kernel(const ChunkBwdArgs a) {
    static_assert(KS == 1 || NC == 4, "");
    extern __shared__ __align__(128) char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    constexpr int kSplit = 8 * KS / NC, kSlice = D / kSplit, kJ = 16 / KS;
    const int lane = threadIdx.x & 31;
    const Roles<NC, 8, 0> role(warp_index());
    const int unit = blockIdx.x / kSplit, dv0 = (blockIdx.x % kSplit) * kSlice;
    const int n = by_length(unit / a.HV, a.num_seqs, a.T, a.cu_seqlens);
    const int hv = unit % a.HV, h = hv / (a.HV / a.H);
    const Seq sq = seq_of(n, a.T, a.cu_seqlens);
    const int steps = (sq.len + BT - 1) / BT * (BT / C);

    if (role.consumer < 0) {
        role.give();
        const int tid = role.prep * 32 + lane;
        for (int i = 0; i < kRaw - 1; ++i) {
            if (i < steps) load_step<kSlice>(sm, a, sq, h, hv, dv0, i, steps - 1 - i, tid);
            cp_async_commit();
        }
        for (int i = 0; i < steps; ++i) {
            const int st = i & 1;
            cp_wait<kRaw - 2>();
            if (i >= kStages) bar_sync(BAR_EMPTY + st, kPrepThreads + 32 * NC);
            bar_sync(BAR_PREP, kPrepThreads);
            prep_planes<T16, kPrepThreads, false>(sm.raw[i % kRaw], sm.prep[st].planes,
                                                  sm.prep[st].decay, a.scale, tid);
            bar_arrive(BAR_FULL + st, kPrepThreads + 32 * NC);
            if (i + kRaw - 1 < steps)
                load_step<kSlice>(sm, a, sq, h, hv, dv0, i + kRaw - 1, steps - kRaw - i, tid);
            cp_async_commit();
        }
        cp_async_wait_all();
        return;
    }

    role.take();
    // this warp's tile of the slice, its first dv column, its part of dk
    const int cw = role.consumer, tile = cw / KS, d0 = dv0 + tile * 16, kh = cw % KS;
    const int k0 = kh * (8 / KS);  // first 16 channels of dk
    const int gr = lane >> 2, tc2 = (lane & 3) * 2;
    const size_t sbase = ((size_t)n * a.HV + hv) * D * D + (size_t)k0 * 16 * D;
    const bool states_in = state_ok(a, a.d_final_state, sbase, DBG_LOAD) &&
                           state_ok(a, a.d_initial_state, sbase, DBG_STORE);
    float S[kJ][4];  // dS^T: rows dv d0 + gr, + 8; columns dk 8j + tc2, + 1 of its part
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        if (a.d_final_state && states_in) {
            const float *p = a.d_final_state + sbase + (size_t)(8 * j + tc2) * D + d0 + gr;
            S[j][0] = p[0];
            S[j][1] = p[D];
            S[j][2] = p[8];
            S[j][3] = p[D + 8];
        } else {
            S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
        }
    }
    const int lrow = (lane & 7) + ((lane >> 4) & 1) * 8, lcol = (lane >> 3) & 1;
    const int trow = lane & 15, tcol = lane >> 4;
    // transposed reads of a [16][16] tile: B fragments of its rows as the summed dimension
    const uint32_t ttile = (uint32_t)(((lane & 7) + ((lane >> 3) & 1) * 8) * 32 + (lane >> 4) * 16);
    const size_t vrow = (size_t)a.HV * D;
    uint16_t *dv_at = (uint16_t *)a.dv + (size_t)sq.row0 * vrow + (size_t)hv * D + d0 + tc2;

    for (int i = 0; i < steps; ++i) {
        const int st = i & 1, step = steps - 1 - i;
        const unsigned slot = (unsigned)(sq.slot0 + step / 4) * a.HV + hv;
        const bool save = dbg_ok(a.dbg, slot, a.units, DBG_STORE);
        if (save && step % 4 == 3)
            store_checkpoint(a.dckpt + slot * kCkptBytes, S, d0 / 16, kh * kJ, lane);
        bar_sync(BAR_FULL + st, kPrepThreads + 32 * NC);
        const Prepared &in = sm.prep[st];
        const uint32_t pl = tc::smem_u32(in.planes);
        constexpr bool kExact = std::is_same<T16, __nv_bfloat16>::value;
        uint32_t ah[4], al[4], oh[4], ol[4], ph[4], plo[4], th[4], tlo[4];
        // do^T as left operand (dv rows, tokens summed): exact in BF16, split in two for FP16
        ldsm4t(oh, tc::smem_u32(sm.dout[i % kRing]) + plane_off(lrow, tile * 2 + lcol));
        const uint32_t tl = tc::smem_u32(sm.tiles[i % kRing]) + ttile;
        ldsm4t(ph, tl + 2 * kTile);
        ldsm4t(plo, tl + 3 * kTile);
        ldsm4t(th, tl);
        ldsm4t(tlo, tl + kTile);
        const float2 b0 = *reinterpret_cast<const float2 *>(&sm.beta[i % kRing][tc2]);
        const float2 b1 = *reinterpret_cast<const float2 *>(&sm.beta[i % kRing][8 + tc2]);
        if (!kExact) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = unpack2<T16>(oh[j]);
                split2(x.x, x.y, oh[j], ol[j]);
            }
        }
        // dn^T = do^T P + dS'^T kd^T, in three chains a tile that are added at the end
        float dn[2][4] = {}, dn2[2][4] = {}, dn3[2][4] = {}, low[2][4];
        auto join_chains = [&] {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    dn[j][p] += dn2[j][p] + dn3[j][p];
                    dn2[j][p] = dn3[j][p] = 0.f;
                }
        };
#pragma unroll
        for (int kk = 0; kk < 8 / KS; ++kk) {
            if (KS == 1 && kk == 4) {  // the halves of dk apart, as where two warps have them
                join_chains();
                take_sum(dn, low);
            }
            uint32_t bh[4], bl[4];
            const uint32_t off = plane_off(lrow, 2 * (k0 + kk) + lcol);
            ldsm4(bh, pl + KD_HI * kPlane + off);
            ldsm4(bl, pl + KD_LO * kPlane + off);
            split_frag(S[2 * kk], S[2 * kk + 1], ah, al);
            mma16816(dn[0], ah, bh[0], bh[1]);
            mma16816(dn[1], ah, bh[2], bh[3]);
            mma16816(dn2[0], ah, bl[0], bl[1]);
            mma16816(dn2[1], ah, bl[2], bl[3]);
            mma16816(dn3[0], al, bh[0], bh[1]);
            mma16816(dn3[1], al, bh[2], bh[3]);
        }
        join_chains();
        if (KS == 1) add_sum(dn, low);
        float4(*join)[2][32] = sm.join[i & 1];
        if (KS == 2) {
            join[cw][0][lane] = make_float4(dn[0][0], dn[0][1], dn[0][2], dn[0][3]);
            join[cw][1][lane] = make_float4(dn[1][0], dn[1][1], dn[1][2], dn[1][3]);
        }
        mma16816(dn2[0], oh, ph[0], ph[1]);
        mma16816(dn2[1], oh, ph[2], ph[3]);
        mma16816(dn3[0], oh, plo[0], plo[1]);
        mma16816(dn3[1], oh, plo[2], plo[3]);
        if (!kExact) {
            mma16816(dn3[0], ol, ph[0], ph[1]);
            mma16816(dn3[1], ol, ph[2], ph[3]);
        }
        if (KS == 2) {
            bar_sync(BAR_JOIN + (cw >> 1), 64);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 x = join[cw ^ 1][j][lane];
                dn[j][0] += x.x; dn[j][1] += x.y; dn[j][2] += x.z; dn[j][3] += x.w;
            }
        }
        join_chains();
        // Y^T = dn^T T
        float y[2][4] = {}, y2[2][4] = {}, y3[2][4] = {};
        split_frag(dn[0], dn[1], ah, al);
        mma16816(y[0], ah, th[0], th[1]);
        mma16816(y[1], ah, th[2], th[3]);
        mma16816(y2[0], ah, tlo[0], tlo[1]);
        mma16816(y2[1], ah, tlo[2], tlo[3]);
        mma16816(y3[0], al, th[0], th[1]);
        mma16816(y3[1], al, th[2], th[3]);
        // dS = diag(2^g_l) dS' + qw^T do - kw^T dv; what needs no Y fills Y's latency
#pragma unroll
        for (int jj = 0; jj < 8 / KS; jj += 2) {
            uint32_t qh[4], ql[4], rh[4], rl[4];
            decay_cols(S, in.decay + 16 * k0, jj, tc2);
            decay_cols(S, in.decay + 16 * k0, jj + 1, tc2);
            const uint32_t o0 = plane_off(trow, 2 * (k0 + jj) + tcol);
            const uint32_t o1 = plane_off(trow, 2 * (k0 + jj) + 2 + tcol);
            ldsm4t(qh, pl + QW_HI * kPlane + o0);
            ldsm4t(rh, pl + QW_HI * kPlane + o1);
            ldsm4t(ql, pl + QW_LO * kPlane + o0);
            ldsm4t(rl, pl + QW_LO * kPlane + o1);
            mma_in<kExact>(S[2 * jj], S[2 * jj + 1], S[2 * jj + 2], S[2 * jj + 3], oh, ol, qh, ql,
                           rh, rl);
        }
        float dv[2][4];  // -dv = -beta Y, the left operand of the state's update
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 b = j ? b1 : b0;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                y[j][p] += y2[j][p] + y3[j][p];
                dv[j][p] = -(p & 1 ? b.y : b.x) * y[j][p];
            }
        }
        split_frag(dv[0], dv[1], ah, al);
#pragma unroll
        for (int jj = 0; jj < 8 / KS; jj += 2) {
            uint32_t wh[4], wl[4], lh[4], ll[4];
            const uint32_t o0 = plane_off(trow, 2 * (k0 + jj) + tcol);
            const uint32_t o1 = plane_off(trow, 2 * (k0 + jj) + 2 + tcol);
            ldsm4t(wh, pl + KW_HI * kPlane + o0);
            ldsm4t(lh, pl + KW_HI * kPlane + o1);
            ldsm4t(wl, pl + KW_LO * kPlane + o0);
            ldsm4t(ll, pl + KW_LO * kPlane + o1);
            mma3x2<true>(S[2 * jj], S[2 * jj + 1], S[2 * jj + 2], S[2 * jj + 3], ah, al, wh, wl, ah,
                         al, lh, ll);
        }
        if (i + kStages < steps) bar_arrive(BAR_EMPTY + st, kPrepThreads + 32 * NC);
        // Y and dv, eight tokens at a time
        auto put = [&](const float (&yj)[4], const float (&x)[4], int j) {
            if (save) store_row_block(a.y + slot * kRowsBytes, yj, (step % 4) * C / 8 + j, d0, lane);
            const uint32_t u = movm_t(pack2<T16>(-x[0], -x[1]));
            const uint32_t w = movm_t(pack2<T16>(-x[2], -x[3]));
            const int t = step * C + 8 * j + gr;
            uint16_t *at = dv_at + (size_t)t * vrow;
            if (t < sq.len &&
                dbg_ok(a.dbg, (size_t)(at - (uint16_t *)a.dv) + 9, a.rows_o * D, DBG_STORE)) {
                *reinterpret_cast<uint32_t *>(at) = u;
                *reinterpret_cast<uint32_t *>(at + 8) = w;
            }
        };
        if (KS == 1) {
            put(y[0], dv[0], 0);
            put(y[1], dv[1], 1);
        } else {
            float yh[4], dh[4];
            half_of(y, kh, yh);
            half_of(dv, kh, dh);
            put(yh, dh, kh);
        }
    }
    if (a.d_initial_state && states_in) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            float *p = a.d_initial_state + sbase + (size_t)(8 * j + tc2) * D + d0 + gr;
            p[0] = S[j][0];
            p[D] = S[j][1];
            p[8] = S[j][2];
            p[D + 8] = S[j][3];
        }
    }
}

template <typename T16, int NC, int KS>
cudaError_t launch(const ChunkBwdArgs &a, int dev, cudaStream_t stream) {
    static volatile int done[kMaxDev];
    const auto kernel = kda_chunk_bwd_state_kernel<T16, NC, KS>;
    const cudaError_t e = ready_once<Roles<NC, 8, 0>>(kernel, (int)sizeof(Smem), dev, done);
    if (e != cudaSuccess) return e;
    const int grid = a.num_seqs * a.HV * (8 * KS / NC);
    kernel<<<grid, Roles<NC, 8, 0>::kThreads, sizeof(Smem), stream>>>(a);
    return cudaGetLastError();
}

template <typename T16>
cudaError_t launch_split(const ChunkBwdArgs &a, int dev, cudaStream_t stream) {
    switch (best_split(a.num_seqs, a.HV, a.cu_seqlens)) {
        case 1: return launch<T16, 8, 1>(a, dev, stream);
        case 2: return launch<T16, 4, 1>(a, dev, stream);
        default: return launch<T16, 4, 2>(a, dev, stream);
    }
}

}  // namespace

cudaError_t launch_bwd_state(const ChunkBwdArgs &a, int dev, cudaStream_t stream) {
    return a.fp16 ? launch_split<__half>(a, dev, stream) : launch_split<__nv_bfloat16>(a, dev, stream);
}

}  // namespace chunk
}  // namespace kda
