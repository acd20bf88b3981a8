// Forward of the gated delta-rule recurrence: one CTA walks one (sequence, value head) in
// steps of 16 tokens (see kda_chunk.cuh for the mathematics).
#include "kda_chunk.cuh"
#include "kda_ops.h"

namespace kda {
namespace chunk {
namespace {

constexpr int kStages = 3;         // prepared stages
constexpr int kRaw = kStages + 2;  // raw input stages: two ahead, and as far back as a stage lives
constexpr int kHalf = 128;         // threads of each half of the preparing warps

// Named barriers; PLANES, FULL, EMPTY + stage.
enum { BAR_PREP = 1, BAR_SCORE = 2, BAR_PLANES = 3, BAR_FULL = 6, BAR_EMPTY = 9 };

struct __align__(128) Prepared {
    char planes[kPlanes * kPlane];
    char t2[2 * kTile];  // hi, lo
    char p[2 * kTile];
    float decay[D];
    int from_start;      // the key plane is k 2^-g (decay after adding), not k 2^(g_l - g)
};

struct __align__(128) Smem {
    Prepared prep[kStages];
    RawStage raw[kRaw];
    uint16_t v[kRaw][C][D];  // rows of the CTA's dv slice, swizzled chunks
    float beta[kRaw][C];
    float a2[2][C][C + 4];   // M diag(beta), two steps' worth
    float a1[2][C][C + 4];   // diag(beta) M
    char t[2 * kTile];       // T hi, lo on the way to the saved tiles
};

template <typename T16, int NC>
__device__ __forceinline__ void load_step(Smem &sm, const ChunkFwdArgs &a, const Seq &sq, int h,
                                          int hv, int dv0, int step, int tid) {
    RawStage &raw = sm.raw[step % kRaw];
    const int c = tid & 15;
#pragma unroll
    for (int i = 0; i < C * 16 / kHalf; ++i) {
        const int row = (tid >> 4) + i * (kHalf / 16), t = step * C + row;
        const bool ok = t < sq.len;
        const size_t tok = (size_t)sq.row0 + (ok ? t : 0);
        const size_t iq = (tok * a.H + h) * D + c * 8, iv = (tok * a.HV + hv) * D;
        cp16z(tc::smem_u32(&raw.q[row][c * 8]), (const uint16_t *)a.q + iq, ok);
        cp16z(tc::smem_u32(&raw.k[row][c * 8]), (const uint16_t *)a.k + iq, ok);
        cp16z(tc::smem_u32(&raw.gate[row][c * 4]), a.gate + iv + c * 4, ok);
        cp16z(tc::smem_u32(&raw.gate[row][64 + c * 4]), a.gate + iv + 64 + c * 4, ok);
        if (c < 2 * NC)
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
                sm.a2[buf][r][s] = x * beta[s];
                sm.a1[buf][r][s] = x * beta[r];
            }
            if (s + 1 < r) {
                sm.a2[buf][r][s + 1] = y * beta[s + 1];
                sm.a1[buf][r][s + 1] = y * beta[r];
            }
        }
    }
}

// Gates so strong that k 2^-g leaves FP32's range inside a step (a channel loses more than
// 2^-96 in 16 tokens): the key plane in its bounded form, the gate replaced by its cumsum ...
template <typename T16>
__device__ __noinline__ void prep_strong(RawStage &raw, Prepared &out, float scale, int tid) {
    prep_planes<T16, kHalf, false>(raw, out.planes, out.decay, scale, tid);
    bar_sync(BAR_PREP, kHalf);
    float acc = 0.f;
    for (int r = 0; r < C; ++r) raw.gate[r][tid] = acc += floor_gate(raw.gate[r][tid]);
}

// ... and M and P pair by pair, one exp2 per (r, s, channel), every exponent <= 0: 17 pairs of
// the rows w and 15 - w a call.  Lane l holds channels 4l .. 4l + 3.
template <typename T16>
__device__ __noinline__ void scores_strong(Smem &sm, const RawStage &raw, const float *beta,
                                           Prepared &out, int buf, float scale, int w, int lane) {
    auto row4 = [&](const uint16_t *p, float (&x)[4]) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p + 4 * lane);
        const float2 lo = unpack2<T16>(u.x), hi = unpack2<T16>(u.y);
        x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
    };
    float q1[4], k1[4], q2[4], k2[4];
    const int r1 = w, r2 = C - 1 - w;
    row4(raw.q[r1], q1);
    row4(raw.k[r1], k1);
    row4(raw.q[r2], q2);
    row4(raw.k[r2], k2);
    const float4 g1 = *reinterpret_cast<const float4 *>(&raw.gate[r1][4 * lane]);
    const float4 g2 = *reinterpret_cast<const float4 *>(&raw.gate[r2][4 * lane]);
    float v[32], lastp = 0.f;
#pragma unroll
    for (int j = 0; j < 17; ++j) {
        const bool first = j <= w;
        const int s = first ? j : j - w - 1;
        float ks[4];
        row4(raw.k[s], ks);
        const float4 gs = *reinterpret_cast<const float4 *>(&raw.gate[s][4 * lane]);
        const float4 gr = first ? g1 : g2;
        const float e[4] = {ex2(gr.x - gs.x) * ks[0], ex2(gr.y - gs.y) * ks[1],
                            ex2(gr.z - gs.z) * ks[2], ex2(gr.w - gs.w) * ks[3]};
        float p = 0.f, m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p += (first ? q1[i] : q2[i]) * e[i];
            m += (first ? k1[i] : k2[i]) * e[i];
        }
        if (j < 16) {
            v[2 * j] = p;
            v[2 * j + 1] = m;
        } else {
            lastp = p;  // the pair (r2, r2): only P has a diagonal
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lastp += __shfl_xor_sync(0xffffffffu, lastp, off);
    const float sum = transpose_sum(v, lane);
    auto put = [&](int r, int s, float x, bool is_p) {
        if (is_p) {  // the entries above the diagonal are zero from the start or from scores()
            const uint32_t b = pack_bf16(x * scale, 0.f) & 0xffffu;
            const float rest = x * scale - __uint_as_float(b << 16);
            reinterpret_cast<uint16_t *>(out.p)[r * C + s] = (uint16_t)b;
            reinterpret_cast<uint16_t *>(out.p + kTile)[r * C + s] =
                (uint16_t)(pack_bf16(rest, 0.f) & 0xffffu);
        } else if (s < r) {
            sm.a2[buf][r][s] = x * beta[s];
            sm.a1[buf][r][s] = x * beta[r];
        }
    };
    const int j = lane >> 1;
    const bool first = j <= w;
    put(first ? r1 : r2, first ? j : j - w - 1, sum, !(lane & 1));
    if (lane == 0) put(r2, r2, lastp, true);
}

// T2 = (I + M diag(beta))^-1 (lanes 0-15, one column each) and T = (I + diag(beta) M)^-1
// (lanes 16-31) by forward substitution in FP32.
__device__ __forceinline__ void solve(Smem &sm, Prepared &out, int buf, int lane) {
    const int c = lane & 15;
    const bool second = lane >= 16;
    const float(*A)[C + 4] = second ? sm.a1[buf] : sm.a2[buf];
    float x[C];
#pragma unroll
    for (int r = 0; r < C; ++r) {
        float s = r == c ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < r; j += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(&A[r][j]);
            s -= a.x * x[j];
            if (j + 1 < r) s -= a.y * x[j + 1];
            if (j + 2 < r) s -= a.z * x[j + 2];
            if (j + 3 < r) s -= a.w * x[j + 3];
        }
        x[r] = s;
    }
    uint16_t *hi = reinterpret_cast<uint16_t *>(second ? sm.t : out.t2);
    uint16_t *lo = hi + C * C;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const uint32_t b = pack_bf16(x[r], 0.f) & 0xffffu;
        hi[r * C + c] = (uint16_t)b;
        lo[r * C + c] =
            (uint16_t)(pack_bf16(x[r] - __uint_as_float(b << 16), 0.f) & 0xffffu);
    }
}

// Whether any lane holds a value that is not finite.
__device__ __forceinline__ bool any_bad(const float (&x)[2][4]) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) s = fmaf(x[j][p], 0.f, s);  // NaN once one is not
    return __any_sync(0xffffffffu, s != 0.f);
}

// acc += X L^T for a lower-triangular [16][16] tile L (hi, lo) where X [16 dv, 16 tokens] has
// values that are not finite: times the zeros above L's diagonal they would spoil tokens
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

template <typename T16, int NC, bool SAVE>
__global__ void __launch_bounds__(kPrepThreads + 32 * NC, 1)
    kda_chunk_fwd_kernel(const ChunkFwdArgs a) {
    extern __shared__ __align__(128) char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    constexpr int kSplit = 8 / NC;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = blockIdx.x / kSplit, dv0 = (blockIdx.x % kSplit) * NC * 16;
    const int n = unit / a.HV, hv = unit - n * a.HV, h = hv / (a.HV / a.H);
    const Seq sq = seq_of(n, a.T, a.cu_seqlens);
    // whole 64-token slots where the backward's buffers are written: rows past the end are
    // computed as zeros, so every row of a slot is defined
    const int steps = SAVE ? (sq.len + BT - 1) / BT * (BT / C) : (sq.len + C - 1) / C;

    // P's entries above the diagonal are never written later
    for (int i = tid; i < kStages * 2 * kTile / 4; i += blockDim.x)
        reinterpret_cast<uint32_t *>(sm.prep[i / (2 * kTile / 4)].p)[i % (2 * kTile / 4)] = 0u;
    __syncthreads();

    if (warp < kPrepWarps) {
        if (NC == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        if (tid < kHalf) {  // raw inputs -> operand planes
            for (int i = 0; i < 2; ++i) {
                if (i < steps) load_step<T16, NC>(sm, a, sq, h, hv, dv0, i, tid);
                cp_async_commit();
            }
            for (int i = 0; i < steps; ++i) {
                const int st = i % kStages;
                Prepared &out = sm.prep[st];
                RawStage &raw = sm.raw[i % kRaw];
                cp_wait<1>();
                // the consumers are done with this stage's previous step (and its values)
                if (i >= kStages) bar_sync(BAR_EMPTY + st, kHalf + 32 * NC);
                bar_sync(BAR_PREP, kHalf);
                if (i + 2 < steps) load_step<T16, NC>(sm, a, sq, h, hv, dv0, i + 2, tid);
                cp_async_commit();
                const bool big = prep_planes<T16, kHalf, true>(raw, out.planes, out.decay, a.scale,
                                                               tid);
                const bool strong = bar_or(BAR_PREP, kHalf, big);
                if (strong) prep_strong<T16>(raw, out, a.scale, tid);
                if (tid == 0) out.from_start = !strong;
                bar_arrive(BAR_PLANES + st, 2 * kHalf);
            }
            cp_async_wait_all();
            return;
        }
        // planes -> scores -> T2 and T
        const int w = warp - kHalf / 32;
        for (int i = 0; i < steps; ++i) {
            const int st = i % kStages;
            Prepared &out = sm.prep[st];
            const float *beta = sm.beta[i % kRaw];
            bar_sync(BAR_PLANES + st, 2 * kHalf);
            if (out.from_start) {
                scores(sm, out, beta, i & 1, w, lane);
            } else {
                scores_strong<T16>(sm, sm.raw[i % kRaw], beta, out, i & 1, a.scale, w, lane);
                scores_strong<T16>(sm, sm.raw[i % kRaw], beta, out, i & 1, a.scale, w + 4, lane);
            }
            bar_sync(BAR_SCORE, kHalf);
            if (w == 0) {
                if (SAVE || lane < 16) solve(sm, out, i & 1, lane);
                __syncwarp();
                bar_arrive(BAR_FULL + st, 32 + 32 * NC);
                if (SAVE && dv0 == 0) {
                    uint4 *to = reinterpret_cast<uint4 *>(
                        a.tiles +
                        (((size_t)(sq.slot0 + i / 4) * a.HV + hv) * 4 + i % 4) * kTilesBytes);
                    const uint4 *t = reinterpret_cast<const uint4 *>(sm.t);
                    const uint4 *p = reinterpret_cast<const uint4 *>(out.p);
                    to[lane] = t[lane];
                    to[32 + lane] = t[32 + lane];
                    to[64 + lane] = p[lane];
                    to[96 + lane] = p[32 + lane];
                    __syncwarp();
                }
            }
        }
        return;
    }

    // ------------------------------------------------------------------ consumers
    if (NC == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    const int cw = warp - kPrepWarps, d0 = dv0 + cw * 16;  // this warp's dv columns
    const int gr = lane >> 2, tc2 = (lane & 3) * 2;
    const size_t sbase = ((size_t)n * a.HV + hv) * D * D;
    float S[16][4];  // S^T: rows d0 + gr, d0 + gr + 8; columns dk 8j + tc2, + 1
    if (a.initial_state) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float *p = a.initial_state + sbase + (size_t)(8 * j + tc2) * D + d0 + gr;
            S[j][0] = p[0];
            S[j][1] = p[D];
            S[j][2] = p[8];
            S[j][3] = p[D + 8];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
    }
    // ldmatrix lane addresses: row-major operand planes and the transposed reads of kd
    const int lrow = (lane & 7) + ((lane >> 4) & 1) * 8, lcol = (lane >> 3) & 1;
    const int trow = lane & 15, tcol = lane >> 4;

    for (int i = 0; i < steps; ++i) {
        const int st = i % kStages;
        if (SAVE && i % 4 == 0)
            store_checkpoint(a.ckpt + ((size_t)(sq.slot0 + i / 4) * a.HV + hv) * kCkptBytes, S, d0,
                             lane);
        bar_sync(BAR_FULL + st, 32 + 32 * NC);
        const Prepared &in = sm.prep[st];
        const uint32_t pl = tc::smem_u32(in.planes);
        float xw[2][4] = {}, xq[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            uint32_t ah[4], al[4], bh[4], bl[4];
            split_frag(S[2 * kk], S[2 * kk + 1], ah, al);
            const uint32_t off = plane_off(lrow, 2 * kk + lcol);
            ldsm4(bh, pl + KW_HI * kPlane + off);
            ldsm4(bl, pl + KW_LO * kPlane + off);
            mma3(xw[0], xw[1], ah, al, bh, bl);
            ldsm4(bh, pl + QW_HI * kPlane + off);
            ldsm4(bl, pl + QW_LO * kPlane + off);
            mma3(xq[0], xq[1], ah, al, bh, bl);
        }
        // R = v - kw S
        uint32_t vr[4];
        {
            // transposed 8x8 blocks (tokens 0-7, dv 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
            const int rr = (lane & 7) + ((lane >> 4) & 1) * 8, cc = (lane >> 3) & 1;
            ldsm4t(vr, tc::smem_u32(sm.v[i % kRaw]) + plane_off(rr, cw * 2 + cc));
        }
        float R[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 x = unpack2<T16>(vr[2 * j]), y = unpack2<T16>(vr[2 * j + 1]);
            R[j][0] = x.x - xw[j][0];
            R[j][1] = x.y - xw[j][1];
            R[j][2] = y.x - xw[j][2];
            R[j][3] = y.y - xw[j][3];
        }
        const uint32_t tl = tile_lane(lane);
        uint32_t ah[4], al[4], bh[4], bl[4];
        float e[2][4] = {};
        if (any_bad(R)) {
            mma_causal(e, R, tc::smem_u32(in.t2), tc::smem_u32(in.t2) + kTile, lane);
        } else {
            split_frag(R[0], R[1], ah, al);
            ldsm4(bh, tc::smem_u32(in.t2) + tl);
            ldsm4(bl, tc::smem_u32(in.t2) + kTile + tl);
            mma3(e[0], e[1], ah, al, bh, bl);
        }
        if (SAVE)
            store_rows(a.e + ((size_t)(sq.slot0 + i / 4) * a.HV + hv) * kRowsBytes, e, (i % 4) * C,
                       d0, lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 b = *reinterpret_cast<const float2 *>(&sm.beta[i % kRaw][8 * j + tc2]);
            e[j][0] *= b.x;
            e[j][1] *= b.y;
            e[j][2] *= b.x;
            e[j][3] *= b.y;
        }
        split_frag(e[0], e[1], ah, al);  // n = beta e
        if (any_bad(e)) {
            mma_causal(xq, e, tc::smem_u32(in.p), tc::smem_u32(in.p) + kTile, lane);
        } else {
            ldsm4(bh, tc::smem_u32(in.p) + tl);
            ldsm4(bl, tc::smem_u32(in.p) + kTile + tl);
            mma3(xq[0], xq[1], ah, al, bh, bl);
        }
        // S' = 2^g_l (S + (k 2^-g)^T n), or with strong gates 2^g_l S + (k 2^(g_l - g))^T n
        auto decayed = [&](int jj) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 d = *reinterpret_cast<const float2 *>(&in.decay[16 * jj + 8 * x + tc2]);
                float(&s)[4] = S[2 * jj + x];
                const float2 u = mul2(make_float2(s[0], s[1]), d);
                const float2 w = mul2(make_float2(s[2], s[3]), d);
                s[0] = u.x; s[1] = u.y; s[2] = w.x; s[3] = w.y;
            }
        };
        const bool from_start = in.from_start;
        if (!from_start) {
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) decayed(jj);
        }
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
            const uint32_t off = plane_off(trow, 2 * jj + tcol);
            ldsm4t(bh, pl + KD_HI * kPlane + off);
            ldsm4t(bl, pl + KD_LO * kPlane + off);
            mma3(S[2 * jj], S[2 * jj + 1], ah, al, bh, bl);
        }
        if (from_start) {
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) decayed(jj);
        }
        if (i + kStages < steps) bar_arrive(BAR_EMPTY + st, kHalf + 32 * NC);
        // o: rows of tokens after the transpose
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t x = movm_t(pack2<T16>(xq[j][0], xq[j][1]));
            const uint32_t y = movm_t(pack2<T16>(xq[j][2], xq[j][3]));
            const int t = i * C + 8 * j + gr;
            if (t < sq.len) {
                const size_t idx = ((size_t)(sq.row0 + t) * a.HV + hv) * D + d0 + tc2;
                if (dbg_ok(a.dbg, idx + 9, a.rows_o * D, DBG_STORE)) {
                    *reinterpret_cast<uint32_t *>((uint16_t *)a.o + idx) = x;
                    *reinterpret_cast<uint32_t *>((uint16_t *)a.o + idx + 8) = y;
                }
            }
        }
    }
    if (a.final_state) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float *p = a.final_state + sbase + (size_t)(8 * j + tc2) * D + d0 + gr;
            p[0] = S[j][0];
            p[D] = S[j][1];
            p[8] = S[j][2];
            p[D + 8] = S[j][3];
        }
    }
}

template <typename T16, int NC, bool SAVE>
cudaError_t launch(const ChunkFwdArgs &a, int dev, cudaStream_t stream) {
    static volatile int done[kMaxDev];
    cudaError_t e =
        smem_limit_once(kda_chunk_fwd_kernel<T16, NC, SAVE>, (int)sizeof(Smem), dev, done);
    if (e != cudaSuccess) return e;
    const int grid = a.num_seqs * a.HV * (8 / NC);
    kda_chunk_fwd_kernel<T16, NC, SAVE>
        <<<grid, kPrepThreads + 32 * NC, sizeof(Smem), stream>>>(a);
    return cudaGetLastError();
}

template <typename T16, bool SAVE>
cudaError_t launch_nc(const ChunkFwdArgs &a, int dev, cudaStream_t stream) {
    const long long heads = (long long)a.num_seqs * a.HV;
    if (heads * 2 > kSMs) return launch<T16, 8, SAVE>(a, dev, stream);
    if (heads * 4 > kSMs) return launch<T16, 4, SAVE>(a, dev, stream);
    return launch<T16, 2, SAVE>(a, dev, stream);
}

}  // namespace
}  // namespace chunk

cudaError_t launch_chunk_fwd(const ChunkFwdArgs &a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool save = a.ckpt != nullptr;
    if (a.fp16)
        return save ? chunk::launch_nc<__half, true>(a, dev, stream)
                    : chunk::launch_nc<__half, false>(a, dev, stream);
    return save ? chunk::launch_nc<__nv_bfloat16, true>(a, dev, stream)
                : chunk::launch_nc<__nv_bfloat16, false>(a, dev, stream);
}

}  // namespace kda
