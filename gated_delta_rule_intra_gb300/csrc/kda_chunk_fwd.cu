// Forward of the gated delta-rule recurrence: one CTA walks one (sequence, value head), or a part
// of its dv columns, in steps of 16 tokens (see kda_chunk.cuh for the mathematics).
//
// Warps have the same four parts as in kda_fast_fwd.cu; three BF16 products take the place of one
// FP16 product.  Bound by the time of a step on one SM: 4.8, 3.3 and 2.7 thousand cycles with
// one, two and four CTAs a head.  In four, two consumer warps share 16 dv columns and have half of
// dk each: their 48 + 24 products a step take a third of the 2.7, the rest is the preparation's
// share of the issue slots (52% taken) and of the shared-memory pipe (61%), which every CTA of a
// head repeats.  B=1 T=32768 H=32: 2.70 ms for 2048 steps; 37 tokens: 7.4 us.
#include <type_traits>

#include "kda_chunk.cuh"
#include "kda_ops.h"

namespace kda {
namespace fast {
cudaError_t launch_fwd(const ChunkFwdArgs &a, int dev, cudaStream_t stream);  // kda_fast_fwd.cu
}  // namespace fast

namespace chunk {
namespace {

constexpr int kStages = 3;         // prepared stages
constexpr int kRaw = kStages + 2;  // raw input stages: two ahead, and as far back as a stage lives
constexpr int kHalf = 128;         // threads that take the scores

// Named barriers; JOIN + pair of consumers that share a tile; PLANES, FULL, EMPTY, SOLVE + stage.
enum {
    BAR_PREP = 0,
    BAR_JOIN = 1,
    BAR_PLANES = 3,
    BAR_FULL = 6,
    BAR_EMPTY = 9,
    BAR_SOLVE = 12
};

struct __align__(128) Prepared {
    char planes[kPlanes * kPlane];
    char t2[2 * kTile];  // hi, lo
    char p[2 * kTile];
    float decay[D];
    int from_start;      // the key plane is k 2^-g (decay after adding), not k 2^(g_l - g)
    int careful;         // gates too strong for that, or inputs that are not finite
};

struct __align__(128) Smem {
    Prepared prep[kStages];
    RawStage raw[kRaw];
    uint16_t v[kRaw][C][D];  // rows of the CTA's dv slice, swizzled chunks
    float beta[kRaw][C];
    float a2[kStages][C][C + 4];  // (M diag(beta))^T
    float a1[kStages][C][C + 4];  // (diag(beta) M)^T
    char t[kStages][2 * kTile];   // T hi, lo on the way to the saved tiles
    int bad[kStages][4];          // whether a warp has seen an input that is not finite
    char out[8][512];             // a consumer's o on its way out
    float4 join[2][4][3][32];     // partial sums of consumers that share a tile, two steps' worth
};

template <int SLICE, int NT>
__device__ __forceinline__ void load_step(Smem &sm, const ChunkFwdArgs &a, const Seq &sq, int h,
                                          int hv, int dv0, int step, int tid) {
    RawStage &raw = sm.raw[step % kRaw];
    const int c = tid & 15;
#pragma unroll
    for (int i = 0; i < C * 16 / NT; ++i) {
        const int row = (tid >> 4) + i * (NT / 16), t = step * C + row;
        const bool ok = t < sq.len && token_ok(a, sq.row0 + t);
        const size_t tok = (size_t)sq.row0 + (ok ? t : 0);
        const size_t iq = (tok * a.H + h) * D + c * 8, iv = (tok * a.HV + hv) * D;
        cp16z(tc::smem_u32(&raw.q[row][c * 8]), (const uint16_t *)a.q + iq, ok);
        cp16z(tc::smem_u32(&raw.k[row][c * 8]), (const uint16_t *)a.k + iq, ok);
        cp16z(tc::smem_u32(&raw.gate[row][c * 4]), a.gate + iv + c * 4, ok);
        cp16z(tc::smem_u32(&raw.gate[row][64 + c * 4]), a.gate + iv + 64 + c * 4, ok);
        if (c < SLICE / 8)
            cp16z(tc::smem_u32(sm.v[step % kRaw]) + plane_off(row, c),
                  (const uint16_t *)a.v + iv + dv0 + c * 8, ok);
        if (c == 0)
            cp4z(tc::smem_u32(&sm.beta[step % kRaw][row]), a.beta + tok * a.HV + hv, ok);
    }
}

// M and P of a step are one product each, M = kw (k 2^-g)^T and P = qw (k 2^-g)^T: the
// exponents cancel in each term and no term is above |q_r k_s|.  One warp an 8-column half.
// The halves' other entries (s > r) may be of any size and are dropped.
__device__ __forceinline__ void scores(Smem &sm, Prepared &out, const float *beta, int buf, int w,
                                       int lane) {
    const bool is_p = w & 1;
    const int nt = w >> 1, m = lane >> 3;
    const uint32_t pl = tc::smem_u32(out.planes);
    const uint32_t left = pl + (is_p ? QW_HI : KW_HI) * kPlane;
    const uint32_t right = pl + (KD_HI + (m >> 1)) * kPlane;
    const int arow = (lane & 7) + (m & 1) * 8;
    float c0[4] = {}, c1[4] = {}, c2[4] = {};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        uint32_t ah[4], al[4], b[4];
        const uint32_t off = plane_off(arow, 2 * kk + (m >> 1));
        ldsm4(ah, left + off);
        ldsm4(al, left + kPlane + off);
        ldsm4(b, right + plane_off(8 * nt + (lane & 7), 2 * kk + (m & 1)));
        mma16816(c0, ah, b[0], b[1]);
        mma16816(c1, ah, b[2], b[3]);
        mma16816(c2, al, b[0], b[1]);
    }
    const int s = 8 * nt + (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 2) + 8 * i;
        float x = c0[2 * i] + (c1[2 * i] + c2[2 * i]);
        float y = c0[2 * i + 1] + (c1[2 * i + 1] + c2[2 * i + 1]);
        if (is_p) {
            uint32_t hi, lo;
            split2(s <= r ? x : 0.f, s + 1 <= r ? y : 0.f, hi, lo);
            *reinterpret_cast<uint32_t *>(out.p + (r * C + s) * 2) = hi;
            *reinterpret_cast<uint32_t *>(out.p + kTile + (r * C + s) * 2) = lo;
        } else {
            if (s < r) {
                sm.a2[buf][s][r] = x * beta[s];
                sm.a1[buf][s][r] = x * beta[r];
            }
            if (s + 1 < r) {
                sm.a2[buf][s + 1][r] = y * beta[s + 1];
                sm.a1[buf][s + 1][r] = y * beta[r];
            }
        }
    }
}

// Gates so strong that k 2^-g leaves FP32's range inside a step (a channel loses more than
// 2^-96 or so in 16 tokens), or keys and gates that are not finite: the key plane is taken
// in its bounded form, and M and P pair by pair, one exp2 per (r, s, channel), every exponent <= 0
// and summed from the pair's own gates.  17 pairs of the rows w and 15 - w a call, each row's from
// its diagonal on.  Lane l holds channels 4l .. 4l + 3.
template <typename T16>
__device__ __forceinline__ void scores_strong(Smem &sm, const RawStage &raw, const float *beta,
                                              Prepared &out, int buf, float scale, int w,
                                              int lane) {
    auto row4 = [&](const uint16_t *p, float (&x)[4]) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p + 4 * lane);
        const float2 lo = unpack2<T16>(u.x), hi = unpack2<T16>(u.y);
        x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
    };
    float4 d = make_float4(0.f, 0.f, 0.f, 0.f);  // the gates behind s up to r
#pragma unroll 1
    for (int j = 0; j < 17; ++j) {
        const int r = j <= w ? w : C - 1 - w, s = j <= w ? w - j : C - j;
        float q[4], k[4], ks[4];
        row4(raw.q[r], q);
        row4(raw.k[r], k);
        row4(raw.k[s], ks);
        if (s == r) d = make_float4(0.f, 0.f, 0.f, 0.f);
        const float e[4] = {ex2(d.x) * ks[0], ex2(d.y) * ks[1], ex2(d.z) * ks[2],
                            ex2(d.w) * ks[3]};
        const float4 g = *reinterpret_cast<const float4 *>(&raw.gate[s][4 * lane]);
        d.x += floor_gate(g.x); d.y += floor_gate(g.y);
        d.z += floor_gate(g.z); d.w += floor_gate(g.w);
        float p = 0.f, m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p += q[i] * e[i];
            m += k[i] * e[i];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            p += __shfl_xor_sync(0xffffffffu, p, off);
            m += __shfl_xor_sync(0xffffffffu, m, off);
        }
        if (lane == 0) {  // P's entries above the diagonal are zero from the start or scores()
            uint32_t hi, lo;
            split2(p * scale, 0.f, hi, lo);
            reinterpret_cast<uint16_t *>(out.p)[r * C + s] = (uint16_t)hi;
            reinterpret_cast<uint16_t *>(out.p + kTile)[r * C + s] = (uint16_t)lo;
            if (s < r) {
                sm.a2[buf][s][r] = m * beta[s];
                sm.a1[buf][s][r] = m * beta[r];
            }
        }
    }
}

// T2 = (I + M diag(beta))^-1 (lanes 0-15, one column each) and T = (I + diag(beta) M)^-1
// (lanes 16-31) by forward substitution in FP32, column by column of the matrix: a found entry
// is taken out of all later rows at once.
__device__ __forceinline__ void solve(Smem &sm, Prepared &out, int buf, int lane) {
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
    uint16_t *hi = reinterpret_cast<uint16_t *>(second ? sm.t[buf] : out.t2);
    uint16_t *lo = hi + C * C;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const uint32_t b = pack_bf16(x[r], 0.f) & 0xffffu;
        hi[r * C + c] = (uint16_t)b;
        lo[r * C + c] =
            (uint16_t)(pack_bf16(x[r] - __uint_as_float(b << 16), 0.f) & 0xffffu);
    }
}

// Whether any value or beta of a step is not finite (128 threads, SLICE columns of values).
template <typename T16, int SLICE>
__device__ __forceinline__ bool not_finite(const uint16_t (*v)[D], const float *beta, int tid) {
    float2 acc = make_float2(0.f, 0.f);
    const float2 zero = acc;
#pragma unroll
    for (int i = 0; i < C * SLICE / 8 / kHalf + (C * SLICE / 8 < kHalf); ++i) {
        const int x = tid + i * kHalf, row = x / (SLICE / 8), c = x % (SLICE / 8);
        if (row < C) {
            const uint4 u =
                *reinterpret_cast<const uint4 *>((const char *)v + plane_off(row, c));
            acc = fma2(unpack2<T16>(u.x), zero, acc);
            acc = fma2(unpack2<T16>(u.y), zero, acc);
            acc = fma2(unpack2<T16>(u.z), zero, acc);
            acc = fma2(unpack2<T16>(u.w), zero, acc);
        }
    }
    if (tid < C) acc.x = fmaf(beta[tid], 0.f, acc.x);
    return acc.x + acc.y != 0.f;  // NaN once one was not finite
}

// acc += X L^T for a lower-triangular [16][16] tile L (hi, lo) where X [16 dv, 16 tokens] may
// have values that are not finite: times the zeros above L's diagonal they would spoil tokens
// before their own.  Each token's column is taken from the tokens up to it alone.
__device__ __forceinline__ void mma_causal(float (&acc)[2][4], const float (&x)[2][4], uint32_t hi,
                                           uint32_t lo, int lane) {
    uint32_t bh[4], bl[4];
    ldsm4(bh, hi + tile_lane(lane));
    ldsm4(bl, lo + tile_lane(lane));
    const int tc2 = (lane & 3) * 2;
#pragma unroll 1
    for (int r = 0; r < C; ++r) {
        float m[2][4], c[2][4] = {};
        uint32_t ah[4], al[4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p) m[j][p] = 8 * j + tc2 + (p & 1) <= r ? x[j][p] : 0.f;
        split_frag(m[0], m[1], ah, al);
        mma3(c[0], c[1], ah, al, bh, bl);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (8 * j + tc2 + (p & 1) == r) acc[j][p] += c[j][p];
    }
}

template <int NJ>
__device__ __forceinline__ void scale_all(float (&S)[NJ][4], float (&n)[2][4], float (&o)[2][4],
                                          float f) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) S[j][p] *= f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            n[j][p] *= f;
            o[j][p] *= f;
        }
}

// One step of a consumer warp's 16 columns of dv: e and o (xq) of its tokens, S updated.
// With KS = 2 the warp has the half `kh` of dk: sums over dk are joined with the partner's in
// shared memory, both warps have e, and o is finished for the tokens 8 kh .. 8 kh + 7.
// One straight run of code, so that the chain R -> e -> n of a tile overlaps other products;
// CAREFUL also takes steps with strong gates or inputs that are not finite.  CKPT: the state's
// operand halves, which the first product needs anyway, are stored as the slot's checkpoint.
template <typename T16, int KS, bool CAREFUL, bool CKPT>
__device__ __forceinline__ void consume(float (&S)[16 / KS][4], float (&xq)[2][4],
                                        float (&e)[2][4], const Prepared &in,
                                        const uint16_t (*v)[D], const float *beta, char *ckpt,
                                        int slice_tile, int tile, int kh,
                                        float4 (*join)[3][32], int warp, int lane) {
    const int k0 = kh * (8 / KS);  // first 16 channels of dk
    const int tc2 = (lane & 3) * 2;
    // ldmatrix lane addresses: row-major operand planes and the transposed reads of kd
    const int lrow = (lane & 7) + ((lane >> 4) & 1) * 8, lcol = (lane >> 3) & 1;
    const int trow = lane & 15, tcol = lane >> 4;
    const uint32_t pl = tc::smem_u32(in.planes), tl = tile_lane(lane);
    float xw[2][4], lw[2][4], lq[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) xw[j][p] = xq[j][p] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 8 / KS; ++kk) {
        if (KS == 1 && kk == 4) {  // the halves of dk apart, as where two warps have them
            take_sum(xw, lw);
            take_sum(xq, lq);
        }
        uint32_t kf[4], kl[4], qh[4], ql[4];
        const uint32_t off = plane_off(lrow, 2 * (k0 + kk) + lcol);
        ldsm4(kf, pl + KW_HI * kPlane + off);
        ldsm4(qh, pl + QW_HI * kPlane + off);
        ldsm4(kl, pl + KW_LO * kPlane + off);
        ldsm4(ql, pl + QW_LO * kPlane + off);
        uint32_t ah[4], al[4];
        split_frag(S[2 * kk], S[2 * kk + 1], ah, al);
        mma3x2<true>(xw[0], xw[1], xq[0], xq[1], ah, al, kf, kl, ah, al, qh, ql);
        if (CKPT) {
            uint4 *p = reinterpret_cast<uint4 *>(ckpt) +
                       (2 * (k0 + kk) * 8 + slice_tile + tile) * 32 + lane;
            p[0] = make_uint4(movm_t(ah[0]), movm_t(al[0]), movm_t(ah[1]), movm_t(al[1]));
            p[8 * 32] = make_uint4(movm_t(ah[2]), movm_t(al[2]), movm_t(ah[3]), movm_t(al[3]));
        }
    }
    if (KS == 1) {
        add_sum(xw, lw);
        add_sum(xq, lq);
    } else {
        auto put = [&](int i, const float (&x)[4]) {
            join[warp][i][lane] = make_float4(x[0], x[1], x[2], x[3]);
        };
        auto add = [&](int i, float (&x)[4]) {
            const float4 y = join[warp ^ 1][i][lane];
            x[0] += y.x; x[1] += y.y; x[2] += y.z; x[3] += y.w;
        };
        put(0, xw[0]);
        put(1, xw[1]);
        float own[4], other[4];
        half_of(xq, kh, own);
        half_of(xq, !kh, other);
        put(2, other);
        bar_sync(BAR_JOIN + (warp >> 1), 64);
        add(0, xw[0]);
        add(1, xw[1]);
        add(2, own);
#pragma unroll
        for (int p = 0; p < 4; ++p) xq[0][p] = xq[1][p] = own[p];
    }
    uint32_t th[4], tlo[4], nh[4], nl[4];
    ldsm4(th, tc::smem_u32(in.t2) + tl);
    ldsm4(tlo, tc::smem_u32(in.t2) + kTile + tl);
    const float2 b[2] = {*reinterpret_cast<const float2 *>(&beta[tc2]),
                         *reinterpret_cast<const float2 *>(&beta[8 + tc2])};
    // transposed 8x8 blocks (tokens 0-7, dv 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
    uint32_t vr[4];
    ldsm4t(vr, tc::smem_u32(v) + plane_off(lrow, tile * 2 + lcol));
    float R[2][4];  // v - kw S
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float2 x = unpack2<T16>(vr[2 * j]), y = unpack2<T16>(vr[2 * j + 1]);
        R[j][0] = x.x - xw[j][0];
        R[j][1] = x.y - xw[j][1];
        R[j][2] = y.x - xw[j][2];
        R[j][3] = y.y - xw[j][3];
        e[j][0] = e[j][1] = e[j][2] = e[j][3] = 0.f;
    }
    if (CAREFUL) {
        mma_causal(e, R, tc::smem_u32(in.t2), tc::smem_u32(in.t2) + kTile, lane);
    } else {
        uint32_t ah[4], al[4];
        float e2[2][4] = {}, e3[2][4] = {};
        split_frag(R[0], R[1], ah, al);
        mma16816(e[0], ah, th[0], th[1]);
        mma16816(e[1], ah, th[2], th[3]);
        mma16816(e2[0], ah, tlo[0], tlo[1]);
        mma16816(e2[1], ah, tlo[2], tlo[3]);
        mma16816(e3[0], al, th[0], th[1]);
        mma16816(e3[1], al, th[2], th[3]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p) e[j][p] += e2[j][p] + e3[j][p];
    }
    float nb[2][4], most = 0.f;  // n = beta e
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            nb[j][p] = e[j][p] * (p & 1 ? b[j].y : b[j].x);
            most = fmaxf(most, fabsf(nb[j][p]));
        }
    // the key plane reaches 2^96: beside n of this size the sums would leave FP32's range
    const bool large = __any_sync(0xffffffffu, most > 0x1p24f);
    if (large) scale_all(S, nb, xq, 0x1p-72f);
    split_frag(nb[0], nb[1], nh, nl);
    if (CAREFUL) mma_causal(xq, nb, tc::smem_u32(in.p), tc::smem_u32(in.p) + kTile, lane);
    // S' = 2^g_l (S + (k 2^-g)^T n), or with strong gates 2^g_l S + (k 2^(g_l - g))^T n
    const bool from_start = !CAREFUL || uniform(in.from_start);
    if (CAREFUL && !from_start) {
#pragma unroll
        for (int jj = 0; jj < 8 / KS; ++jj) decay_cols(S, in.decay + 16 * k0, jj, tc2);
    }
#pragma unroll
    for (int jj = 0; jj < 8 / KS; jj += 2) {
        uint32_t bh[4], bl[4], ch[4], cl[4];
        const uint32_t o0 = plane_off(trow, 2 * (k0 + jj) + tcol);
        const uint32_t o1 = plane_off(trow, 2 * (k0 + jj) + 2 + tcol);
        ldsm4t(bh, pl + KD_HI * kPlane + o0);
        ldsm4t(ch, pl + KD_HI * kPlane + o1);
        ldsm4t(bl, pl + KD_LO * kPlane + o0);
        ldsm4t(cl, pl + KD_LO * kPlane + o1);
        mma3x2<true>(S[2 * jj], S[2 * jj + 1], S[2 * jj + 2], S[2 * jj + 3], nh,
                     nl, bh, bl, nh, nl, ch, cl);
    }
    // o = qw S + P n
    if (!CAREFUL) {
        ldsm4(th, tc::smem_u32(in.p) + tl);
        ldsm4(tlo, tc::smem_u32(in.p) + kTile + tl);
        if (KS == 1) {
            mma3(xq[0], xq[1], nh, nl, th, tlo);
        } else {
            const uint32_t h0 = kh ? th[2] : th[0], h1 = kh ? th[3] : th[1];
            const uint32_t l0 = kh ? tlo[2] : tlo[0], l1 = kh ? tlo[3] : tlo[1];
            mma16816(xq[0], nh, h0, h1);
            mma16816(xq[0], nh, l0, l1);
            mma16816(xq[0], nl, h0, h1);
        }
    }
    if (from_start) {
#pragma unroll
        for (int jj = 0; jj < 8 / KS; ++jj) decay_cols(S, in.decay + 16 * k0, jj, tc2);
    }
    if (large) scale_all(S, nb, xq, 0x1p72f);
}

// NW consumer warps, KS for each 16 columns of dv: a head takes 8 KS / NW CTAs.  Four of these
// are bound by the preparation, which then has eight warps instead of four.
template <int NW, int KS> using Roles = chunk::Roles<NW, 4 * KS + 4, 4>;

// Eight tokens of o and, for the backward, of e on their way out.
template <typename T16>
__device__ __forceinline__ void finish(const ChunkFwdArgs &a, const float (&o)[4],
                                       const float (&e)[4], bool save, unsigned slot, int step,
                                       int j, uint16_t *o_at, size_t orow, int len, int d0,
                                       int lane) {
    if (save) store_row_block(a.e + slot * kRowsBytes, e, (step % 4) * C / 8 + j, d0, lane);
    const uint32_t x = movm_t(pack2<T16>(o[0], o[1])), y = movm_t(pack2<T16>(o[2], o[3]));
    const int tok = step * C + 8 * j + (lane >> 2);
    uint16_t *at = o_at + (size_t)tok * orow + (lane & 3) * 2;
    if (tok < len && dbg_ok(a.dbg, (size_t)(at - (uint16_t *)a.o) + 9, a.rows_o * D, DBG_STORE)) {
        *reinterpret_cast<uint32_t *>(at) = x;
        *reinterpret_cast<uint32_t *>(at + 8) = y;
    }
}

template <typename T16, int NW, int KS, bool SAVE>
__global__ void __launch_bounds__(Roles<NW, KS>::kThreads, 1)
    kda_chunk_fwd_kernel(const ChunkFwdArgs a) {
    wait_for_previous();
    constexpr int kSlice = 16 * NW / KS, kSplit = D / kSlice, kJ = 16 / KS;
    constexpr int kPrep = 128 * KS;  // threads that prepare operands
    extern __shared__ __align__(128) char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int lane = threadIdx.x & 31;
    const Roles<NW, KS> role(warp_index());
    const int unit = blockIdx.x / kSplit, dv0 = (blockIdx.x % kSplit) * kSlice;
    const int n = by_length(unit / a.HV, a.num_seqs, a.T, a.cu_seqlens);
    const int hv = unit % a.HV, h = hv / (a.HV / a.H);
    const Seq sq = seq_of(n, a.T, a.cu_seqlens);
    // whole 64-token slots where the backward's buffers are written: rows past the end are
    // computed as zeros, so every row of a slot is defined
    const int steps = SAVE ? (sq.len + BT - 1) / BT * (BT / C) : (sq.len + C - 1) / C;

    // P's entries above the diagonal are never written later
    for (int i = threadIdx.x; i < kStages * 2 * kTile / 4; i += blockDim.x)
        reinterpret_cast<uint32_t *>(sm.prep[i / (2 * kTile / 4)].p)[i % (2 * kTile / 4)] = 0u;
    __syncthreads();

    if (role.consumer < 0) {
        role.give();
        if (role.prep >= 0 && role.prep < 4 * KS) {  // raw inputs -> operand planes
            const int tid = role.prep * 32 + lane;
            for (int i = 0; i < 2; ++i) {
                if (i < steps) load_step<kSlice, kPrep>(sm, a, sq, h, hv, dv0, i, tid);
                cp_async_commit();
            }
            for (int i = 0; i < steps; ++i) {
                const int st = i % kStages;
                Prepared &out = sm.prep[st];
                const RawStage &raw = sm.raw[i % kRaw];
                cp_wait<1>();
                // the consumers are done with this stage's previous step (and its values)
                if (i >= kStages) bar_sync(BAR_EMPTY + st, kPrep + 32 * NW);
                bar_sync(BAR_PREP, kPrep);
                const bool big =
                    prep_planes<T16, kPrep, true>(raw, out.planes, out.decay, a.scale, tid);
                const bool strong = bar_or(BAR_PREP, kPrep, big);
                if (strong)
                    prep_planes<T16, kPrep, false>(raw, out.planes, out.decay, a.scale, tid);
                if (tid == 0) out.from_start = !strong;
                bar_arrive(BAR_PLANES + st, kPrep + kHalf);
                if (i + 2 < steps) load_step<kSlice, kPrep>(sm, a, sq, h, hv, dv0, i + 2, tid);
                cp_async_commit();
            }
            cp_async_wait_all();
            return;
        }
        if (role.prep >= 0) {
            // planes -> scores
            const int w = role.prep - 4 * KS, tid = w * 32 + lane;
            for (int i = 0; i < steps; ++i) {
                const int st = i % kStages;
                Prepared &out = sm.prep[st];
                const int buf = st;
                const float *beta = sm.beta[i % kRaw];
                bar_sync(BAR_PLANES + st, kPrep + kHalf);
                if (uniform(out.from_start)) {
                    scores(sm, out, beta, buf, w, lane);
                } else {
                    scores_strong<T16>(sm, sm.raw[i % kRaw], beta, out, buf, a.scale, w, lane);
                    scores_strong<T16>(sm, sm.raw[i % kRaw], beta, out, buf, a.scale, w + 4, lane);
                }
                const bool bad = __any_sync(
                    0xffffffffu, not_finite<T16, kSlice>(sm.v[i % kRaw], beta, tid));
                if (lane == 0) sm.bad[buf][w] = bad;
                bar_arrive(BAR_SOLVE + buf, kHalf + 32);
            }
            return;
        }
        if (role.solver >= 0) {  // scores -> T2 and T
            const int st = role.solver;  // a stage each
            Prepared &out = sm.prep[st];
            for (int i = st; st < kStages && i < steps; i += kStages) {
                bar_sync(BAR_SOLVE + st, kHalf + 32);
                const uint4 *p = reinterpret_cast<const uint4 *>(out.p);
                const uint4 p0 = p[lane], p1 = p[32 + lane];
                if (lane == 0) {
                    const int *bad = sm.bad[st];
                    out.careful = bad[0] || bad[1] || bad[2] || bad[3] || !out.from_start;
                }
                if (SAVE || lane < 16) solve(sm, out, st, lane);
                __syncwarp();
                bar_arrive(BAR_FULL + st, 32 + 32 * NW);
                const size_t unit_at = (size_t)(sq.slot0 + i / 4) * a.HV + hv;
                if (SAVE && dv0 == 0 && dbg_ok(a.dbg, unit_at, a.units, DBG_STORE)) {
                    uint4 *to =
                        reinterpret_cast<uint4 *>(a.tiles + (unit_at * 4 + i % 4) * kTilesBytes);
                    const uint4 *t = reinterpret_cast<const uint4 *>(sm.t[st]);
                    to[lane] = t[lane];
                    to[32 + lane] = t[32 + lane];
                    to[64 + lane] = p0;
                    to[96 + lane] = p1;
                    __syncwarp();
                }
            }
            return;
        }
        return;
    }

    // ------------------------------------------------------------------ consumers
    role.take();
    // this warp's tiles of the slice, its first dv column, its part of dk
    const int cw = role.consumer, tile = cw / KS, d0 = dv0 + tile * 16, kh = cw % KS;
    const int gr = lane >> 2, tc2 = (lane & 3) * 2;
    const size_t sbase = ((size_t)n * a.HV + hv) * D * D + (size_t)kh * (D / KS) * D;
    const bool states_in = state_ok(a, a.initial_state, sbase, DBG_LOAD) &&
                           state_ok(a, a.final_state, sbase, DBG_STORE);
    float S[kJ][4];  // S^T: rows d0 + gr, + 8; columns dk 8j + tc2, + 1 of its part
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
        if (a.initial_state && states_in) {
            const float *p =
                a.initial_state + sbase + (size_t)(8 * j + tc2) * D + d0 + gr;
            S[j][0] = p[0];
            S[j][1] = p[D];
            S[j][2] = p[8];
            S[j][3] = p[D + 8];
        }
    }

    const size_t orow = (size_t)a.HV * D;
    uint16_t *o_at = (uint16_t *)a.o + (size_t)sq.row0 * orow + (size_t)hv * D + d0;

    for (int i = 0; i < steps; ++i) {
        const int st = i % kStages;
        const unsigned slot = (unsigned)(sq.slot0 + i / 4) * a.HV + hv;
        float xq[2][4], e[2][4];
        bar_sync(BAR_FULL + st, 32 + 32 * NW);
        const Prepared &in = sm.prep[st];
        const uint16_t(*v)[D] = sm.v[i % kRaw];
        const float *beta = sm.beta[i % kRaw];
        char *ckpt = SAVE ? a.ckpt + slot * kCkptBytes : nullptr;
        // tiles of 16 dv columns: of the CTA's slice for v, of the head for the checkpoint
        auto run = [&](auto with_care, auto keep) {
            consume<T16, KS, decltype(with_care)::value, decltype(keep)::value>(
                S, xq, e, in, v, beta, ckpt, dv0 / 16, tile, kh, sm.join[i & 1], cw, lane);
        };
        const bool save = SAVE && dbg_ok(a.dbg, slot, a.units, DBG_STORE);
        const bool keep = save && i % 4 == 0;
        const bool careful = uniform(in.careful);
        if (!careful) {
            if (keep)
                run(std::false_type{}, std::integral_constant<bool, SAVE>{});
            else
                run(std::false_type{}, std::false_type{});
        } else {
            if (keep) store_checkpoint(ckpt, S, d0 / 16, kh * kJ, lane);
            run(std::true_type{}, std::false_type{});
        }
        if (i + kStages < steps) bar_arrive(BAR_EMPTY + st, kPrep + 32 * NW);
        if (KS == 2) {  // the tokens that this warp has finished
            float eh[4], oh[4];
            half_of(e, kh, eh);
            half_of(xq, kh && careful, oh);
            finish<T16>(a, oh, eh, save, slot, i, kh, o_at, orow, sq.len, d0, lane);
            continue;
        }
        if (save)
            store_rows(a.e + slot * kRowsBytes, e, (i % 4) * C, d0, lane);
        uint32_t ow[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            ow[2 * j] = pack2<T16>(xq[j][0], xq[j][1]);
            ow[2 * j + 1] = pack2<T16>(xq[j][2], xq[j][3]);
        }
        store_out(sm.out[cw], ow, (char *)(o_at + (size_t)i * C * orow), orow * 2,
                      sq.len - i * C, (char *)a.o, a.rows_o * D * 2, a.dbg, lane);
    }
    if (a.final_state && states_in) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            float *p = a.final_state + sbase + (size_t)(8 * j + tc2) * D + d0 + gr;
            p[0] = S[j][0];
            p[D] = S[j][1];
            p[8] = S[j][2];
            p[D + 8] = S[j][3];
        }
    }
}

template <typename T16, int NW, int KS, bool SAVE>
cudaError_t launch(const ChunkFwdArgs &a, int dev, cudaStream_t stream) {
    static volatile int done[kMaxDev];
    const auto kernel = kda_chunk_fwd_kernel<T16, NW, KS, SAVE>;
    const cudaError_t e = ready_once<Roles<NW, KS>>(kernel, (int)sizeof(Smem), dev, done);
    if (e != cudaSuccess) return e;
    const int grid = a.num_seqs * a.HV * (8 * KS / NW);
    return launch_early(kernel, grid, Roles<NW, KS>::kThreads, sizeof(Smem), stream, a);
}

template <typename T16, bool SAVE>
cudaError_t launch_split(const ChunkFwdArgs &a, int dev, cudaStream_t stream) {
    switch (best_split(a.num_seqs, a.HV, a.cu_seqlens)) {
        case 1: return launch<T16, 8, 1, SAVE>(a, dev, stream);
        case 2: return launch<T16, 4, 1, SAVE>(a, dev, stream);
        default: return launch<T16, 4, 2, SAVE>(a, dev, stream);
    }
}

}  // namespace
}  // namespace chunk

cudaError_t launch_chunk_fwd(const ChunkFwdArgs &a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (a.fast) return fast::launch_fwd(a, dev, stream);
    const bool save = a.ckpt != nullptr;
    if (a.fp16)
        return save ? chunk::launch_split<__half, true>(a, dev, stream)
                    : chunk::launch_split<__half, false>(a, dev, stream);
    return save ? chunk::launch_split<__nv_bfloat16, true>(a, dev, stream)
                : chunk::launch_split<__nv_bfloat16, false>(a, dev, stream);
}

}  // namespace kda
