// Backward of the gated delta-rule recurrence, second pass: dq, dk, dgate and dbeta of every
// 64-token slot of every head at once, from the state at the slot's start (saved by the
// forward), the state's gradient at its end, e and Y (first pass).
//
// Eight warps own 16 dk channels each and hold S [16 dk, 128 dv] in registers: a step of 16
// tokens is
//   F (forwards):  dq = scale 2^g (do S^T),  dk += -beta 2^g (Y S^T),  S <- 2^g_l S + kd^T (beta e)
//   R (backwards): dk += beta 2^(g_l - g) (e dS'^T),  dS <- 2^g_l dS' + qw^T do - kw^T (beta Y)
// with e and Y known, so nothing is solved, every product is the warp's own (the accumulators
// of S are the left operand's fragments of the products that sum over dv), and what is left
// inside a step is the 16x16 triangle of pairs, taken with one exp2 per (r, s, channel):
//   a[r,s] = scale beta_s do_r.e_s,  b[r,s] = -beta_r beta_s Y_r.e_s  (s <= r, s < r)
//   dq_r += a k_s E,  dk_r += b k_s E,  dk_s += (a q_r + b k_r) E,  E = 2^(g_r - g_s)
// (the pair (t, t) carries no gate: dq_t += a k_t, dk_t += a q_t, apart from x below).
// dbeta_t = Y_t.e_t.  Every term carries 2^(G_r - G_s) of the whole-sequence cumulative gate,
// so with x_t = q dq_t + k (dk as row - dk as column), dgate_t = ln2 (sum of x over the slot's
// tokens from t on + sum_dv S' dS' at the slot's end).
#include <type_traits>

#include "kda_chunk.cuh"
#include "kda_ops.h"

namespace kda {
namespace chunk {

cudaError_t launch_bwd_state(const ChunkBwdArgs &a, int dev, cudaStream_t stream);

namespace {

constexpr int kThreads = 256;
constexpr int QS = D + 8;   // row strides in shared memory: the fragment reads (8 channels of
constexpr int GS = D + 4;   // every second token) fall into different banks

struct __align__(128) Smem {
    char e[kRowsBytes], y[kRowsBytes];  // hi and lo planes, 8x8 blocks
    char dout[kRowsBytes];              // the same; BF16 has no lo plane
    uint16_t q[BT][QS], k[BT][QS];
    float g[BT][GS];                    // cumulative inside each 16-token step
    float beta[BT];
    float a[4][C][C], b[4][C][C];
    float x[3][C][D];                   // dq, dk as row, dk as column of a step
    float col2[C][D];                   // dk as column from rows 11 .. 15
    float tail[D];                      // sum_dv S' dS' at the slot's end
};

__device__ __forceinline__ uint32_t block_addr(uint32_t base, int rb, int cb, int lane) {
    return base + (uint32_t)((rb * 16 + cb) * 128 + (lane & 7) * 16);
}

template <typename T16> struct In {
    static constexpr bool exact = std::is_same<T16, __nv_bfloat16>::value;
};

// (c0, c1) += A B^T with A hi/lo and B's blocks: hi, and lo unless B is exact.
template <bool LO>
__device__ __forceinline__ void mma_b(float (&c0)[4], float (&c1)[4], const uint32_t (&ah)[4],
                                      const uint32_t (&al)[4], const uint32_t (&bh)[4],
                                      const uint32_t (&bl)[4]) {
    mma16816(c0, ah, bh[0], bh[1]);
    mma16816(c1, ah, bh[2], bh[3]);
    mma16816(c0, al, bh[0], bh[1]);
    mma16816(c1, al, bh[2], bh[3]);
    if (LO) {
        mma16816(c0, ah, bl[0], bl[1]);
        mma16816(c1, ah, bl[2], bl[3]);
    }
}

template <typename T16> __device__ __forceinline__ float one(uint16_t x);
template <> __device__ __forceinline__ float one<__nv_bfloat16>(uint16_t x) {
    return __uint_as_float((uint32_t)x << 16);
}
template <> __device__ __forceinline__ float one<__half>(uint16_t x) {
    return __half2float(*reinterpret_cast<const __half *>(&x));
}
template <typename T16> __device__ __forceinline__ uint16_t to16(float x) {
    return (uint16_t)(pack2<T16>(x, 0.f) & 0xffffu);
}

// Pairs (r, s), R0 <= r < R1, s < r, of one channel.
template <typename T16, int R0, int R1>
__device__ __forceinline__ void pairs(Smem &sm, int j, int ch) {
    float g[R1], k[R1], col[R1] = {};
#pragma unroll
    for (int s = 0; s < R1; ++s) {
        g[s] = sm.g[j * C + s][ch];
        k[s] = one<T16>(sm.k[j * C + s][ch]);
    }
#pragma unroll
    for (int r = R0; r < R1; ++r) {
        const float q = one<T16>(sm.q[j * C + r][ch]);
        float dq = 0.f, dk = 0.f;
#pragma unroll
        for (int s = 0; s < r; ++s) {
            const float a = sm.a[j][r][s], b = sm.b[j][r][s];
            const float e = ex2(g[r] - g[s]), ke = k[s] * e;
            dq += a * ke;
            dk += b * ke;
            col[s] += (a * q + b * k[r]) * e;
        }
        sm.x[0][r][ch] += dq;
        sm.x[1][r][ch] += dk;
    }
#pragma unroll
    for (int s = 0; s < R1; ++s) {
        if (R0 == 0)
            sm.x[2][s][ch] += col[s];
        else
            sm.col2[s][ch] = col[s];
    }
}

template <typename T16>
__global__ void __launch_bounds__(kThreads, 1) kda_chunk_bwd_kernel(const ChunkBwdArgs a) {
    extern __shared__ __align__(128) char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    constexpr bool kLo = !In<T16>::exact;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, tc2 = (lane & 3) * 2;
    const int c0 = warp * 16;  // this warp's channels
    const uint32_t se = tc::smem_u32(sm.e), sy = tc::smem_u32(sm.y), so = tc::smem_u32(sm.dout);
    const long long units = (long long)a.slots * a.HV;

    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int slot = (int)(u / a.HV), hv = (int)(u - (long long)slot * a.HV);
        const int h = hv / (a.HV / a.H);
        // the slot's sequence and its first token there
        int n, t0, len;
        long long row0;
        if (a.cu_seqlens) {
            int lo = 0, hi = a.num_seqs - 1;
            while (lo < hi) {  // the last sequence whose slots begin at or before this one
                const int mid = (lo + hi + 1) / 2;
                if (seq_of(mid, a.T, a.cu_seqlens).slot0 <= slot) lo = mid; else hi = mid - 1;
            }
            n = lo;
        } else {
            n = slot / ((a.T + BT - 1) / BT);
        }
        const Seq sq = seq_of(n, a.T, a.cu_seqlens);
        t0 = (slot - sq.slot0) * BT;
        len = sq.len;
        row0 = sq.row0 + t0;
        if (t0 < 0 || t0 >= len) continue;  // no tokens here (the same for every thread)
        const int rows = min(BT, len - t0);
        const size_t su = (size_t)u;

        // ---- loads
        for (int i = tid; i < (int)kRowsBytes / 16; i += kThreads) {
            cp16z(se + i * 16, a.e + su * kRowsBytes + i * 16, true);
            cp16z(sy + i * 16, a.y + su * kRowsBytes + i * 16, true);
        }
        for (int i = tid; i < BT * 16; i += kThreads) {
            const int r = i >> 4, c = i & 15;
            const bool ok = r < rows;
            const size_t tok = (size_t)(row0 + (ok ? r : 0));
            cp16z(tc::smem_u32(&sm.q[r][c * 8]), (const uint16_t *)a.q + (tok * a.H + h) * D + c * 8,
                  ok);
            cp16z(tc::smem_u32(&sm.k[r][c * 8]), (const uint16_t *)a.k + (tok * a.H + h) * D + c * 8,
                  ok);
            const size_t iv = (tok * a.HV + hv) * D;
            cp16z(tc::smem_u32(&sm.g[r][c * 4]), a.gate + iv + c * 4, ok);
            cp16z(tc::smem_u32(&sm.g[r][64 + c * 4]), a.gate + iv + 64 + c * 4, ok);
            char *to = sm.dout + ((r >> 3) * 16 + c) * 128 + (r & 7) * 16;
            const uint16_t *from = (const uint16_t *)a.dout + iv + c * 8;
            if (!kLo) {
                cp16z(tc::smem_u32(to), from, ok);
            } else {
                uint4 x = make_uint4(0u, 0u, 0u, 0u), hi, lo;
                if (ok) x = *reinterpret_cast<const uint4 *>(from);
                float2 f;
                f = unpack2<T16>(x.x); split2(f.x, f.y, hi.x, lo.x);
                f = unpack2<T16>(x.y); split2(f.x, f.y, hi.y, lo.y);
                f = unpack2<T16>(x.z); split2(f.x, f.y, hi.z, lo.z);
                f = unpack2<T16>(x.w); split2(f.x, f.y, hi.w, lo.w);
                *reinterpret_cast<uint4 *>(to) = hi;
                *reinterpret_cast<uint4 *>(to + kRowPlane) = lo;
            }
        }
        if (tid < BT) sm.beta[tid] = tid < rows ? a.beta[(size_t)(row0 + tid) * a.HV + hv] : 0.f;
        cp_async_commit();
        float S[16][4];  // rows dk c0 + gr, + 8; columns dv 8j + tc2, + 1
        auto load_state = [&](const char *base, int j, float (&x)[4]) {
            const char *p = base + su * kCkptBytes + ((size_t)(c0 / 8) * 16 + j) * 128 + lane * 4;
            const uint32_t h0 = *reinterpret_cast<const uint32_t *>(p);
            const uint32_t h1 = *reinterpret_cast<const uint32_t *>(p + 16 * 128);
            const uint32_t l0 = *reinterpret_cast<const uint32_t *>(p + D * D * 2);
            const uint32_t l1 = *reinterpret_cast<const uint32_t *>(p + D * D * 2 + 16 * 128);
            x[0] = __uint_as_float(h0 << 16) + __uint_as_float(l0 << 16);
            x[1] = __uint_as_float(h0 & 0xffff0000u) + __uint_as_float(l0 & 0xffff0000u);
            x[2] = __uint_as_float(h1 << 16) + __uint_as_float(l1 << 16);
            x[3] = __uint_as_float(h1 & 0xffff0000u) + __uint_as_float(l1 & 0xffff0000u);
        };
#pragma unroll
        for (int j = 0; j < 16; ++j) load_state(a.ckpt, j, S[j]);
        cp_async_wait_all();
        __syncthreads();

        // ---- cumulative gate inside each step, and the pair coefficients
        for (int i = tid; i < 4 * D; i += kThreads) {
            const int ch = i & (D - 1), j = i / D;
            float acc = 0.f;
#pragma unroll
            for (int r = 0; r < C; ++r) {
                acc += floor_gate(sm.g[j * C + r][ch]);
                sm.g[j * C + r][ch] = acc;
            }
        }
        {
            const int j = warp & 3;  // warps 0-3: do.e, warps 4-7: Y.e of step j
            const uint32_t left = warp < 4 ? so : sy;
            const bool left_lo = warp >= 4 || kLo;
            float c[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t ah[4], al[4] = {0u, 0u, 0u, 0u}, bh[4], bl[4];
                const int m = lane >> 3;
                const uint32_t ao = block_addr(left, 2 * j + (m & 1), 2 * kk + (m >> 1), lane);
                const uint32_t bo = block_addr(se, 2 * j + (m >> 1), 2 * kk + (m & 1), lane);
                ldsm4(ah, ao);
                if (left_lo) ldsm4(al, ao + kRowPlane);
                ldsm4(bh, bo);
                ldsm4(bl, bo + kRowPlane);
                mma3(c[0], c[1], ah, al, bh, bl);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int r = gr + (p >> 1) * 8, s = 8 * i + tc2 + (p & 1);
                    const float bs = sm.beta[j * C + s];
                    if (warp < 4) {
                        sm.a[j][r][s] = a.scale * bs * c[i][p];
                    } else {
                        sm.b[j][r][s] = -sm.beta[j * C + r] * bs * c[i][p];
                        const int t = j * C + r;
                        if (r == s && t < rows)
                            ((uint16_t *)a.dbeta)[(size_t)(row0 + t) * a.HV + hv] =
                                to16<T16>(c[i][p]);
                    }
                }
        }
        __syncthreads();

        // this thread's elements of a step: channels c0 + gr, + 8 (i), tokens tc2, tc2 + 1,
        // 8 + tc2, 9 + tc2 (p) -- the fragments' and the accumulators' common layout
        auto token = [&](int p) { return tc2 + (p & 1) + (p >> 1) * 8; };
        float fq[4][2][4], fk[4][2][4];  // [step][channel][token]

        // ---- F
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float cq[2][4] = {}, cy[2][4] = {};
            const int m = lane >> 3;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t ah[4], al[4], bh[4], bl[4];
                split_frag(S[2 * kk], S[2 * kk + 1], ah, al);
                const uint32_t off = block_addr(0, 2 * j + (m >> 1), 2 * kk + (m & 1), lane);
                ldsm4(bh, so + off);
                if (kLo) ldsm4(bl, so + off + kRowPlane);
                mma_b<kLo>(cq[0], cq[1], ah, al, bh, bl);
                ldsm4(bh, sy + off);
                ldsm4(bl, sy + off + kRowPlane);
                mma_b<true>(cy[0], cy[1], ah, al, bh, bl);
            }
            float kd[2][4], dec[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ch = c0 + gr + 8 * i;
                const float gl = sm.g[j * C + C - 1][ch];
                dec[i] = ex2(gl);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int t = j * C + token(p);
                    const float g = sm.g[t][ch], up = ex2(g), bt = sm.beta[t];
                    kd[i][p] = bt * one<T16>(sm.k[t][ch]) * ex2(gl - g);
                    fq[j][i][p] = a.scale * up * cq[p >> 1][2 * i + (p & 1)];
                    fk[j][i][p] = -bt * up * cy[p >> 1][2 * i + (p & 1)];
                }
            }
            uint32_t ah[4], al[4];
            split2(kd[0][0], kd[0][1], ah[0], al[0]);
            split2(kd[1][0], kd[1][1], ah[1], al[1]);
            split2(kd[0][2], kd[0][3], ah[2], al[2]);
            split2(kd[1][2], kd[1][3], ah[3], al[3]);
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    S[2 * jj + i][0] *= dec[0];
                    S[2 * jj + i][1] *= dec[0];
                    S[2 * jj + i][2] *= dec[1];
                    S[2 * jj + i][3] *= dec[1];
                }
                uint32_t bh[4], bl[4];
                const uint32_t off = block_addr(se, 2 * j + (m & 1), 2 * jj + (m >> 1), lane);
                ldsm4t(bh, off);
                ldsm4t(bl, off + kRowPlane);
                mma3(S[2 * jj], S[2 * jj + 1], ah, al, bh, bl);
            }
        }
        // ---- the state's gradient at the slot's end, and sum_dv S' dS'
        {
            float t0s = 0.f, t1s = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float x[4];
                load_state(a.dckpt, j, x);
                t0s += S[j][0] * x[0] + S[j][1] * x[1];
                t1s += S[j][2] * x[2] + S[j][3] * x[3];
#pragma unroll
                for (int p = 0; p < 4; ++p) S[j][p] = x[p];
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                t0s += __shfl_xor_sync(0xffffffffu, t0s, off);
                t1s += __shfl_xor_sync(0xffffffffu, t1s, off);
            }
            if ((lane & 3) == 0) {
                sm.tail[c0 + gr] = t0s;
                sm.tail[c0 + gr + 8] = t1s;
            }
        }
        // ---- R, and each step's triangle and outputs
        float carry = 0.f;
#pragma unroll
        for (int jr = 0; jr < 4; ++jr) {
            const int j = 3 - jr, m = lane >> 3;
            float cd[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t ah[4], al[4], bh[4], bl[4];
                split_frag(S[2 * kk], S[2 * kk + 1], ah, al);
                const uint32_t off = block_addr(se, 2 * j + (m >> 1), 2 * kk + (m & 1), lane);
                ldsm4(bh, off);
                ldsm4(bl, off + kRowPlane);
                mma_b<true>(cd[0], cd[1], ah, al, bh, bl);
            }
            float qw[2][4], kw[2][4], dec[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ch = c0 + gr + 8 * i;
                const float gl = sm.g[j * C + C - 1][ch];
                dec[i] = ex2(gl);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int t = j * C + token(p);
                    const float g = sm.g[t][ch], up = ex2(g), bt = sm.beta[t];
                    qw[i][p] = a.scale * up * one<T16>(sm.q[t][ch]);
                    kw[i][p] = -bt * up * one<T16>(sm.k[t][ch]);
                    sm.x[0][token(p)][ch] = fq[j][i][p];
                    sm.x[1][token(p)][ch] = fk[j][i][p];
                    sm.x[2][token(p)][ch] = bt * ex2(gl - g) * cd[p >> 1][2 * i + (p & 1)];
                }
            }
            if (j > 0) {
                uint32_t ah[4], al[4], wh[4], wl[4];
                split2(qw[0][0], qw[0][1], ah[0], al[0]);
                split2(qw[1][0], qw[1][1], ah[1], al[1]);
                split2(qw[0][2], qw[0][3], ah[2], al[2]);
                split2(qw[1][2], qw[1][3], ah[3], al[3]);
                split2(kw[0][0], kw[0][1], wh[0], wl[0]);
                split2(kw[1][0], kw[1][1], wh[1], wl[1]);
                split2(kw[0][2], kw[0][3], wh[2], wl[2]);
                split2(kw[1][2], kw[1][3], wh[3], wl[3]);
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        S[2 * jj + i][0] *= dec[0];
                        S[2 * jj + i][1] *= dec[0];
                        S[2 * jj + i][2] *= dec[1];
                        S[2 * jj + i][3] *= dec[1];
                    }
                    uint32_t bh[4], bl[4];
                    const uint32_t off = block_addr(0, 2 * j + (m & 1), 2 * jj + (m >> 1), lane);
                    ldsm4t(bh, so + off);
                    if (kLo) ldsm4t(bl, so + off + kRowPlane);
                    mma_b<kLo>(S[2 * jj], S[2 * jj + 1], ah, al, bh, bl);
                    ldsm4t(bh, sy + off);
                    ldsm4t(bl, sy + off + kRowPlane);
                    mma3(S[2 * jj], S[2 * jj + 1], wh, wl, bh, bl);
                }
            }
            __syncthreads();
            const int ch = tid & (D - 1);
            if (warp < 4)
                pairs<T16, 0, 11>(sm, j, ch);
            else
                pairs<T16, 11, 16>(sm, j, ch);
            __syncthreads();
            if (warp < 4) {
                if (jr == 0) carry = sm.tail[ch];
#pragma unroll
                for (int tt = C - 1; tt >= 0; --tt) {
                    const int t = j * C + tt;
                    const float q = one<T16>(sm.q[t][ch]), k = one<T16>(sm.k[t][ch]);
                    float dq = sm.x[0][tt][ch], dk = sm.x[1][tt][ch];
                    const float dkc = sm.x[2][tt][ch] + sm.col2[tt][ch];
                    carry += q * dq + k * (dk - dkc);
                    // the pair (t, t) has no gate: its shares of x would cancel
                    const float diag = sm.a[j][tt][tt];
                    dq += diag * k;
                    dk += dkc + diag * q;
                    if (t < rows) {
                        const size_t tok = (size_t)(row0 + t), iv = (tok * a.HV + hv) * D + ch;
                        if (dbg_ok(a.dbg, iv, a.rows_o * D, DBG_STORE)) {
                            ((uint16_t *)a.dgate)[iv] = to16<T16>(LN2 * carry);
                            if (a.dq_hv) {
                                a.dq_hv[iv] = dq;
                                a.dk_hv[iv] = dk;
                            } else {
                                ((uint16_t *)a.dq)[iv] = to16<T16>(dq);
                                ((uint16_t *)a.dk)[iv] = to16<T16>(dk);
                            }
                        }
                    }
                }
            }
            __syncthreads();
        }
    }
}

// dq and dk of a q/k head: the sum over its value heads, in head order.
template <typename T16>
__global__ void __launch_bounds__(256) kda_chunk_bwd_heads_kernel(const ChunkBwdArgs a) {
    const int G = a.HV / a.H;
    const size_t n = a.rows_o / G * (D / 4);
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * n) return;
    const bool second = i >= n;
    const size_t e = second ? i - n : i, row = e / (D / 4), c = e % (D / 4);
    const size_t tok = row / a.H, h = row % a.H;
    if (a.cu_seqlens) {  // tokens in no sequence have no gradient
        const long long t = (long long)tok;
        if (t < a.cu_seqlens[0] || t >= a.cu_seqlens[a.num_seqs]) return;
    }
    const float4 *from = reinterpret_cast<const float4 *>(second ? a.dk_hv : a.dq_hv) +
                         (tok * a.HV + h * G) * (D / 4) + c;
    float4 s = from[0];
    for (int j = 1; j < G; ++j) {
        const float4 x = from[(size_t)j * (D / 4)];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    uint2 o;
    o.x = pack2<T16>(s.x, s.y);
    o.y = pack2<T16>(s.z, s.w);
    reinterpret_cast<uint2 *>(second ? a.dk : a.dq)[e] = o;
}

template <typename T16>
cudaError_t launch(const ChunkBwdArgs &a, int dev, cudaStream_t stream) {
    cudaError_t e = launch_bwd_state(a, dev, stream);
    if (e != cudaSuccess) return e;
    const long long units = (long long)a.slots * a.HV;
    if (units == 0) return cudaSuccess;
    static volatile int done[kMaxDev];
    e = smem_limit_once(kda_chunk_bwd_kernel<T16>, (int)sizeof(Smem), dev, done);
    if (e != cudaSuccess) return e;
    kda_chunk_bwd_kernel<T16><<<(unsigned)(units < kSMs ? units : kSMs), kThreads, sizeof(Smem),
                                stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || !a.dq_hv) return e;
    const size_t n = 2 * (a.rows_o / (a.HV / a.H)) * (D / 4);
    kda_chunk_bwd_heads_kernel<T16><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace chunk

cudaError_t launch_chunk_bwd(const ChunkBwdArgs &a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return a.fp16 ? chunk::launch<__half>(a, dev, stream)
                  : chunk::launch<__nv_bfloat16>(a, dev, stream);
}

}  // namespace kda
