// Backward of the gated delta-rule recurrence, second pass: dq, dk, dgate and dbeta of every
// 64-token slot of every head at once, from the state at the slot's start (saved by the
// forward), the state's gradient at its end, e and Y (first pass).
//
// Eight warps own 16 dk channels each and hold S [16 dk, 128 dv], or its gradient, in registers.
// A step of 16 tokens is, with e and Y known (nothing is solved),
//   R (backwards): dk_col = beta 2^-g (2^g_l (e dS'^T) + qw^T G1 - (beta kw)^T G2)
//                  dS <- 2^g_l dS' + qw^T do - (beta kw)^T Y
//   F (forwards):  dq = scale 2^g (do S^T + G1 (beta k 2^-g)),
//                  dk_row = -beta 2^g (Y S^T + G2 (beta k 2^-g)),
//                  S <- 2^g_l (S + (beta k 2^-g)^T e)
// where G1[r,s] = do_r.e_s and G2[r,s] = Y_r.e_s (s < r) carry the step's own pairs, whose decay
// 2^(g_r - g_s) is the product of the two sides' factors; dk = dk_row + dk_col, dbeta_t = Y_t.e_t.
// (The pair (t, t) has no decay: scale beta_t do_t.e_t times k_t and q_t, added at the end.)
// Every product is the warp's own: the accumulators of S are the left operand's fragments of
// the products that sum over dv, and a thread's elements of q, k and g, of the left operands
// that sum over tokens and of the results are the same (channel, token) pairs.
//
// Every term carries 2^(G_r - G_s) of the whole-sequence cumulative gate, so with
// x_t = q dq_t + k (dk_row - dk_col)_t the gate's gradient falls by ln2 x_t from a token to the
// next; at a slot's first token it is ln2 sum_dv S dS.
//
// B=8 T=2048 H=16 FP16: 600 us for 4096 slots, 45 thousand cycles each on one SM: three products
// for each of kda_fast_bwd.cu's, whose comment tells what bounds them.
#include <type_traits>

#include "kda_chunk.cuh"
#include "kda_ops.h"

namespace kda {
namespace fast {
cudaError_t launch_bwd(const ChunkBwdArgs &a, int dev, cudaStream_t stream);  // kda_fast_bwd.cu
}  // namespace fast

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
    float beta[BT], diag[BT];           // diag: do_t.e_t
    char g1[4][2 * kTile], g2[4][2 * kTile];  // hi, lo of each step, zero from the diagonal on
    float col[4][8][kThreads];          // dk_col from R to F, each thread's own
    char out[3][kThreads / 32][512];    // a warp's dq, dk, dgate of a step on their way out
};

__device__ __forceinline__ uint32_t block_addr(uint32_t base, int rb, int cb, int lane) {
    return base + (uint32_t)((rb * 16 + cb) * 128 + (lane & 7) * 16);
}

template <typename T16> struct In {
    static constexpr bool exact = std::is_same<T16, __nv_bfloat16>::value;
};

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

// A thread's elements of a step: channels gr, gr + 8 (i) of its warp's 16, tokens tc2, tc2 + 1,
// 8 + tc2, 9 + tc2 (p).
struct Elems {
    float v[2][4];
};
__device__ __forceinline__ int token_of(int p, int tc2) { return tc2 + (p & 1) + (p >> 1) * 8; }

// The elements as a left operand [16 channels, 16 tokens].
__device__ __forceinline__ void split_elems(const Elems &x, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(x.v[0][0], x.v[0][1], hi[0], lo[0]);
    split2(x.v[1][0], x.v[1][1], hi[1], lo[1]);
    split2(x.v[0][2], x.v[0][3], hi[2], lo[2]);
    split2(x.v[1][2], x.v[1][3], hi[3], lo[3]);
}

// q or k of a step (row-major rows of QS elements).
template <typename T16>
__device__ __forceinline__ Elems load_elems(const uint16_t (*rows)[QS], int c0, int lane) {
    uint32_t r[4];
    ldsm4t(r, tc::smem_u32(&rows[(lane & 7) + ((lane >> 4) & 1) * 8][c0 + ((lane >> 3) & 1) * 8]));
    Elems x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T16>(r[i]);
        x.v[i & 1][(i >> 1) * 2] = f.x;
        x.v[i & 1][(i >> 1) * 2 + 1] = f.y;
    }
    return x;
}

__device__ __forceinline__ void decay_rows(float (&S)[16][4], float d0, float d1) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float2 u = mul2(make_float2(S[j][0], S[j][1]), make_float2(d0, d0));
        const float2 w = mul2(make_float2(S[j][2], S[j][3]), make_float2(d1, d1));
        S[j][0] = u.x; S[j][1] = u.y; S[j][2] = w.x; S[j][3] = w.y;
    }
}

// S[16 channels, 128 dv] += A [16 channels, 16 tokens] B, B the step's rows of a block layout.
__device__ __forceinline__ void add_rows(float (&S)[16][4], const uint32_t (&ah)[4],
                                         const uint32_t (&al)[4], uint32_t rows, int j, int lane) {
    const int m = lane >> 3;
#pragma unroll
    for (int jj = 0; jj < 8; jj += 2) {
        uint32_t bh[4], bl[4], ch[4], cl[4];
        const uint32_t o0 = block_addr(rows, 2 * j + (m & 1), 2 * jj + (m >> 1), lane);
        ldsm4t(bh, o0);
        ldsm4t(ch, o0 + 2 * 128);
        ldsm4t(bl, o0 + kRowPlane);
        ldsm4t(cl, o0 + 2 * 128 + kRowPlane);
        mma3x2<true>(S[2 * jj], S[2 * jj + 1], S[2 * jj + 2], S[2 * jj + 3], ah, al, bh, bl, ah, al,
                     ch, cl);
    }
}

// A step's pairs where k 2^-g would leave FP32's range: one exp2 per (r, s, channel), the
// thread's tokens as rows (dq, dk_row; add to what is there) or as columns (dk_col).
template <typename T16>
__device__ __noinline__ void pairs_strong(Smem &sm, int j, int c0, int lane, float scale,
                                          bool columns, Elems &x, Elems &y) {
    auto tile = [](const char *t, int r, int s) {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(t) + r * C + s;
        return __uint_as_float((uint32_t)h[0] << 16) + __uint_as_float((uint32_t)h[C * C] << 16);
    };
    const int gr = lane >> 2, tc2 = (lane & 3) * 2;
    for (int i = 0; i < 2; ++i) {
        const int ch = c0 + gr + 8 * i;
        for (int p = 0; p < 4; ++p) {
            const int t = token_of(p, tc2);
            const float gt = sm.g[j * C + t][ch];
            float u = 0.f, w = 0.f;
            if (!columns) {
                for (int s = 0; s < t; ++s) {
                    const float kb = sm.beta[j * C + s] * one<T16>(sm.k[j * C + s][ch]) *
                                     ex2(gt - sm.g[j * C + s][ch]);
                    u += tile(sm.g1[j], t, s) * kb;
                    w += tile(sm.g2[j], t, s) * kb;
                }
                x.v[i][p] += scale * u;
                y.v[i][p] -= sm.beta[j * C + t] * w;
            } else {
                for (int r = t + 1; r < C; ++r) {
                    const float q = scale * one<T16>(sm.q[j * C + r][ch]);
                    const float k = sm.beta[j * C + r] * one<T16>(sm.k[j * C + r][ch]);
                    u += (tile(sm.g1[j], r, t) * q - tile(sm.g2[j], r, t) * k) *
                         ex2(sm.g[j * C + r][ch] - gt);
                }
                x.v[i][p] += sm.beta[j * C + t] * u;
            }
        }
    }
}

template <typename T16>
__global__ void __launch_bounds__(kThreads, 1) kda_chunk_bwd_kernel(const ChunkBwdArgs a) {
    extern __shared__ __align__(128) char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    constexpr bool kLo = !In<T16>::exact;
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int gr = lane >> 2, tc2 = (lane & 3) * 2, m = lane >> 3;
    const int c0 = warp * 16;  // this warp's channels
    const uint32_t se = tc::smem_u32(sm.e), sy = tc::smem_u32(sm.y), so = tc::smem_u32(sm.dout);
    // lanes' offsets of a [16][16] tile as right operand: rows as columns, or rows summed over
    const uint32_t tn = tile_lane(lane);
    const uint32_t tt = (uint32_t)(((lane & 7) + ((lane >> 3) & 1) * 8) * 32 + (lane >> 4) * 16);
    // a unit's saved blocks take 104 KB, so that their number is far below 2^31
    const unsigned units = (unsigned)a.slots * a.HV;
    const size_t orow = (size_t)a.HV * D;

    Where next = locate(a, blockIdx.x);
    for (unsigned u = blockIdx.x; u < units; u += gridDim.x) {
        const long long row0 = next.row0;
        const unsigned after = u + gridDim.x;
        const int rows = next.rows, h = next.h, hv = next.hv;
        if (after < units) next = locate(a, after);
        if (rows <= 0) continue;  // no tokens here (the same for every thread)
        const size_t su = (size_t)u;

        // ---- loads
        for (int i = tid; i < (int)kRowsBytes / 16; i += kThreads) {
            cp16z(se + i * 16, a.e + su * kRowsBytes + i * 16, true);
            cp16z(sy + i * 16, a.y + su * kRowsBytes + i * 16, true);
        }
        for (int i = tid; i < BT * 16; i += kThreads) {
            const int r = i >> 4, c = i & 15;
            const bool ok = r < rows && token_ok(a, row0 + r);
            const size_t tok = (size_t)(row0 + (ok ? r : 0));
            cp16z(tc::smem_u32(&sm.q[r][c * 8]), (const uint16_t *)a.q + (tok * a.H + h) * D + c * 8,
                  ok);
            cp16z(tc::smem_u32(&sm.k[r][c * 8]), (const uint16_t *)a.k + (tok * a.H + h) * D + c * 8,
                  ok);
            const size_t iv = (tok * a.HV + hv) * D;
            cp16z(tc::smem_u32(&sm.g[r][c * 4]), a.gate + iv + c * 4, ok);
            cp16z(tc::smem_u32(&sm.g[r][64 + c * 4]), a.gate + iv + 64 + c * 4, ok);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // do: eight rows at a time, whose pieces share no banks
            const int r = 16 * x + (warp >> 2) * 8 + (lane & 7), c = (warp & 3) * 4 + (lane >> 3);
            const bool ok = r < rows && token_ok(a, row0 + r);
            char *to = sm.dout + ((r >> 3) * 16 + c) * 128 + (r & 7) * 16;
            const uint16_t *from = (const uint16_t *)a.dout +
                                   ((size_t)(row0 + (ok ? r : 0)) * a.HV + hv) * D + c * 8;
            if (!kLo) {
                cp16z(tc::smem_u32(to), from, ok);
            } else {
                uint4 v = make_uint4(0u, 0u, 0u, 0u), hi, lo;
                if (ok) v = *reinterpret_cast<const uint4 *>(from);
                float2 f;
                f = unpack2<T16>(v.x); split2(f.x, f.y, hi.x, lo.x);
                f = unpack2<T16>(v.y); split2(f.x, f.y, hi.y, lo.y);
                f = unpack2<T16>(v.z); split2(f.x, f.y, hi.z, lo.z);
                f = unpack2<T16>(v.w); split2(f.x, f.y, hi.w, lo.w);
                *reinterpret_cast<uint4 *>(to) = hi;
                *reinterpret_cast<uint4 *>(to + kRowPlane) = lo;
            }
        }
        if (tid < BT)
            sm.beta[tid] = tid < rows && token_ok(a, row0 + tid) ? a.beta[(size_t)(row0 + tid) * a.HV + hv] : 0.f;
        cp_async_commit();
        float S[16][4];  // rows dk c0 + gr, + 8; columns dv 8j + tc2, + 1
        // 16 dv columns of a checkpoint (see store_checkpoint()): tiles 2x and 2x + 1 of S
        auto load_state = [&](const char *base, int x, float (&l)[4], float (&r)[4]) {
            const uint4 *p = reinterpret_cast<const uint4 *>(base + su * kCkptBytes) +
                             ((c0 / 8) * 8 + x) * 32 + lane;
            const uint4 u = p[0], w = p[8 * 32];
            auto sum = [](uint32_t h, uint32_t lo, float &first, float &second) {
                first = __uint_as_float(h << 16) + __uint_as_float(lo << 16);
                second = __uint_as_float(h & 0xffff0000u) + __uint_as_float(lo & 0xffff0000u);
            };
            sum(u.x, u.y, l[0], l[1]);
            sum(w.x, w.y, l[2], l[3]);
            sum(u.z, u.w, r[0], r[1]);
            sum(w.z, w.w, r[2], r[3]);
        };
#pragma unroll
        for (int x = 0; x < 8; ++x) load_state(a.dckpt, x, S[2 * x], S[2 * x + 1]);
        cp_async_wait_all();
        __syncthreads();

        // ---- cumulative gate inside each step, and the pairs' products
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
#pragma unroll 4
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t ah[4], al[4] = {0u, 0u, 0u, 0u}, bh[4], bl[4];
                const uint32_t ao = block_addr(left, 2 * j + (m & 1), 2 * kk + (m >> 1), lane);
                const uint32_t bo = block_addr(se, 2 * j + (m >> 1), 2 * kk + (m & 1), lane);
                ldsm4(ah, ao);
                if (left_lo) ldsm4(al, ao + kRowPlane);
                ldsm4(bh, bo);
                ldsm4(bl, bo + kRowPlane);
                mma3(c[0], c[1], ah, al, bh, bl);
            }
            char *to = warp < 4 ? sm.g1[j] : sm.g2[j];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; p += 2) {
                    const int r = gr + p * 4, s = 8 * i + tc2, t = j * C + r;
                    uint32_t hi, lo;
                    split2(s < r ? c[i][p] : 0.f, s + 1 < r ? c[i][p + 1] : 0.f, hi, lo);
                    *reinterpret_cast<uint32_t *>(to + (r * C + s) * 2) = hi;
                    *reinterpret_cast<uint32_t *>(to + kTile + (r * C + s) * 2) = lo;
                    if (r == s || r == s + 1) {
                        const float d = r == s ? c[i][p] : c[i][p + 1];
                        if (warp < 4)
                            sm.diag[t] = d;
                        else if (t < rows && token_ok(a, row0 + t))
                            put_dbeta(a, (size_t)(row0 + t) * a.HV + hv, d, to16<T16>(d));
                    }
                }
        }
        __syncthreads();

        // the next unit's inputs are asked into L2 while the loads' queue is empty
        if (after < units) {
            const size_t nu = (size_t)after;
            if (tid == 0) {
                tc::prefetch_l2(a.dckpt + nu * kCkptBytes, (uint32_t)kCkptBytes);
                tc::prefetch_l2(a.e + nu * kRowsBytes, (uint32_t)kRowsBytes);
                tc::prefetch_l2(a.y + nu * kRowsBytes, (uint32_t)kRowsBytes);
                tc::prefetch_l2(a.ckpt + nu * kCkptBytes, (uint32_t)kCkptBytes);
            }
            prefetch_rows(a, next, tid, kThreads);
        }
        // ---- R
#pragma unroll 1
        for (int j = 3; j >= 0; --j) {
            float cd[2][4] = {}, cd2[2][4] = {}, cd3[2][4] = {};  // three chains a tile
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t ah[4], al[4], bh[4], bl[4];
                const uint32_t off = block_addr(se, 2 * j + (m >> 1), 2 * kk + (m & 1), lane);
                ldsm4(bh, off);
                ldsm4(bl, off + kRowPlane);
                split_frag(S[2 * kk], S[2 * kk + 1], ah, al);
                mma16816(cd[0], ah, bh[0], bh[1]);
                mma16816(cd[1], ah, bh[2], bh[3]);
                mma16816(cd2[0], ah, bl[0], bl[1]);
                mma16816(cd2[1], ah, bl[2], bl[3]);
                mma16816(cd3[0], al, bh[0], bh[1]);
                mma16816(cd3[1], al, bh[2], bh[3]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int p = 0; p < 4; ++p) cd[x][p] += cd2[x][p] + cd3[x][p];
            const Elems q = load_elems<T16>(&sm.q[j * C], c0, lane);
            const Elems k = load_elems<T16>(&sm.k[j * C], c0, lane);
            Elems qw, kw, g;
            float gl[2], big = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ch = c0 + gr + 8 * i;
                gl[i] = sm.g[j * C + C - 1][ch];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int t = j * C + token_of(p, tc2);
                    g.v[i][p] = sm.g[t][ch];
                    const float up = ex2(g.v[i][p]);
                    qw.v[i][p] = a.scale * up * q.v[i][p];
                    kw.v[i][p] = -sm.beta[t] * up * k.v[i][p];
                }
                big = fmaxf(big, -gl[i]);
            }
            uint32_t ah[4], al[4], wh[4], wl[4];
            split_elems(qw, ah, al);
            split_elems(kw, wh, wl);
            const bool strong = __any_sync(0xffffffffu, big > 96.f);
            Elems col;
            if (!strong) {
                uint32_t bh[4], bl[4];
                const float d0 = ex2(gl[0]), d1 = ex2(gl[1]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    cd[x][0] *= d0; cd[x][1] *= d0; cd[x][2] *= d1; cd[x][3] *= d1;
                }
                ldsm4t(bh, tc::smem_u32(sm.g1[j]) + tt);
                ldsm4t(bl, tc::smem_u32(sm.g1[j]) + kTile + tt);
                mma3(cd[0], cd[1], ah, al, bh, bl);
                ldsm4t(bh, tc::smem_u32(sm.g2[j]) + tt);
                ldsm4t(bl, tc::smem_u32(sm.g2[j]) + kTile + tt);
                mma3(cd[0], cd[1], wh, wl, bh, bl);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float x = strong ? gl[i] - g.v[i][p] : -g.v[i][p];
                    col.v[i][p] = sm.beta[j * C + token_of(p, tc2)] * ex2(x) *
                                  cd[p >> 1][2 * i + (p & 1)];
                }
            if (strong) {
                Elems x = col;
                pairs_strong<T16>(sm, j, c0, lane, a.scale, true, x, x);
                col = x;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) sm.col[j][4 * i + p][tid] = col.v[i][p];
            decay_rows(S, ex2(gl[0]), ex2(gl[1]));
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) {  // + qw^T do - (beta kw)^T Y
                uint32_t bh[4], bl[4], yh[4], yl[4];
                float t0[4] = {}, t1[4] = {};
                const uint32_t off = block_addr(0, 2 * j + (m & 1), 2 * jj + (m >> 1), lane);
                ldsm4t(bh, so + off);
                ldsm4t(yh, sy + off);
                if (kLo) ldsm4t(bl, so + off + kRowPlane);
                ldsm4t(yl, sy + off + kRowPlane);
                mma3x2<kLo>(t0, t1, S[2 * jj], S[2 * jj + 1], ah, al, bh, bl, wh, wl, yh, yl);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    S[2 * jj][p] += t0[p];
                    S[2 * jj + 1][p] += t1[p];
                }
            }
        }
        // ---- the state at the slot's start, and sum_dv S dS there
        float carry[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x[2][4];
            load_state(a.ckpt, i, x[0], x[1]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float(&s)[4] = S[2 * i + y];
                carry[0] += s[0] * x[y][0] + s[1] * x[y][1];
                carry[1] += s[2] * x[y][2] + s[3] * x[y][3];
#pragma unroll
                for (int p = 0; p < 4; ++p) s[p] = x[y][p];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            carry[i] += __shfl_xor_sync(0xffffffffu, carry[i], 1);
            carry[i] += __shfl_xor_sync(0xffffffffu, carry[i], 2);
        }
        // ---- F, and the outputs
        const size_t out_at = (size_t)row0 * orow + (size_t)hv * D + c0;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            float cq[2][4] = {}, cy[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t ah[4], al[4], bh[4], bl[4];
                uint32_t yh[4], yl[4];
                const uint32_t off = block_addr(0, 2 * j + (m >> 1), 2 * kk + (m & 1), lane);
                ldsm4(bh, so + off);
                ldsm4(yh, sy + off);
                if (kLo) ldsm4(bl, so + off + kRowPlane);
                ldsm4(yl, sy + off + kRowPlane);
                split_frag(S[2 * kk], S[2 * kk + 1], ah, al);
                mma3x2<kLo>(cq[0], cq[1], cy[0], cy[1], ah, al, bh, bl, ah, al, yh, yl);
            }
            const Elems q = load_elems<T16>(&sm.q[j * C], c0, lane);
            const Elems k = load_elems<T16>(&sm.k[j * C], c0, lane);
            Elems kd, g;
            float gl[2], big = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                gl[i] = sm.g[j * C + C - 1][c0 + gr + 8 * i];
                big = fmaxf(big, -gl[i]);
            }
            const bool strong = __any_sync(0xffffffffu, big > 96.f);
            // the keys' factors from the middle of the step's decay on: 2^-g itself reaches 2^96,
            // beside which large values would leave FP32's range
            const float mid[2] = {strong ? 0.f : 0.5f * gl[0], strong ? 0.f : 0.5f * gl[1]};
            const float m0 = ex2(mid[0]), m1 = ex2(mid[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int t = j * C + token_of(p, tc2);
                    g.v[i][p] = sm.g[t][c0 + gr + 8 * i];
                    kd.v[i][p] = sm.beta[t] * k.v[i][p] *
                                 ex2((strong ? gl[i] : mid[i]) - g.v[i][p]);
                }
            uint32_t ah[4], al[4];
            split_elems(kd, ah, al);
            if (!strong) {
                uint32_t bh[4], bl[4];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        cq[x][p] *= p < 2 ? m0 : m1;
                        cy[x][p] *= p < 2 ? m0 : m1;
                    }
                decay_rows(S, m0, m1);
                ldsm4(bh, tc::smem_u32(sm.g1[j]) + tn);
                ldsm4(bl, tc::smem_u32(sm.g1[j]) + kTile + tn);
                mma3(cq[0], cq[1], ah, al, bh, bl);
                ldsm4(bh, tc::smem_u32(sm.g2[j]) + tn);
                ldsm4(bl, tc::smem_u32(sm.g2[j]) + kTile + tn);
                mma3(cy[0], cy[1], ah, al, bh, bl);
                add_rows(S, ah, al, se, j, lane);
                decay_rows(S, ex2(gl[0] - mid[0]), ex2(gl[1] - mid[1]));
            } else {
                decay_rows(S, ex2(gl[0]), ex2(gl[1]));
                add_rows(S, ah, al, se, j, lane);
            }
            Elems dq, dk;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float up = ex2(g.v[i][p] - mid[i]);
                    dq.v[i][p] = a.scale * up * cq[p >> 1][2 * i + (p & 1)];
                    dk.v[i][p] = -sm.beta[j * C + token_of(p, tc2)] * up *
                                 cy[p >> 1][2 * i + (p & 1)];
                }
            if (strong) {
                Elems x = dq, y = dk;
                pairs_strong<T16>(sm, j, c0, lane, a.scale, false, x, y);
                dq = x;
                dk = y;
            }
            // the gate's gradient: carry less the x of the tokens before
            Elems dg;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x[4];
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    x[p] = q.v[i][p] * dq.v[i][p] +
                           k.v[i][p] * (dk.v[i][p] - sm.col[j][4 * i + p][tid]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float pair = x[2 * half] + x[2 * half + 1];
                    float incl = pair;  // over the four lanes of the channel
                    float y = __shfl_up_sync(0xffffffffu, incl, 1, 4);
                    if ((lane & 3) >= 1) incl += y;
                    y = __shfl_up_sync(0xffffffffu, incl, 2, 4);
                    if ((lane & 3) >= 2) incl += y;
                    const float before = incl - pair;
                    dg.v[i][2 * half] = LN2 * (carry[i] - before);
                    dg.v[i][2 * half + 1] = LN2 * (carry[i] - before - x[2 * half]);
                    carry[i] -= __shfl_sync(0xffffffffu, incl, 3, 4);
                }
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int t = j * C + token_of(p, tc2);
                const float d = a.scale * sm.beta[t] * sm.diag[t];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    dq.v[i][p] += d * k.v[i][p];
                    dk.v[i][p] += sm.col[j][4 * i + p][tid] + d * q.v[i][p];
                }
            }
            auto put = [&](void *out, int which, const Elems &x) {
                uint32_t w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    w[y] = pack2<T16>(x.v[y & 1][y & 2], x.v[y & 1][(y & 2) + 1]);
                store_out(sm.out[which][warp], w,
                          (char *)((uint16_t *)out + out_at + (size_t)j * C * orow), orow * 2,
                          rows - j * C, (char *)out, a.rows_o * D * 2, a.dbg, lane);
            };
            if (!a.gates32) {
                put(a.dgate, 0, dg);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int t = j * C + token_of(p, tc2);
                        const size_t at = out_at + (size_t)t * orow + 8 * i + gr;
                        if (t < rows && dbg_ok(a.dbg, at, a.rows_o * D, DBG_STORE))
                            ((float *)a.dgate)[at] = dg.v[i][p];
                    }
            }
            if (!a.dq_hv) {
                put(a.dq, 1, dq);
                put(a.dk, 2, dk);
            } else {  // summed over the head's value heads afterwards, in FP32
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int t = j * C + token_of(p, tc2);
                        const size_t at = out_at + (size_t)t * orow + 8 * i + gr;
                        if (t < rows && dbg_ok(a.dbg, at, a.rows_o * D, DBG_STORE)) {
                            a.dq_hv[at] = dq.v[i][p];
                            a.dk_hv[at] = dk.v[i][p];
                        }
                    }
            }
        }
        __syncthreads();
    }
}

// dq and dk of a q/k head: the sum over its value heads, in head order.
template <typename T16>
__global__ void __launch_bounds__(256) kda_chunk_bwd_heads_kernel(const ChunkBwdArgs a) {
    wait_for_previous();
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
    const size_t last = (tok * a.HV + h * G + G - 1) * (D / 4) + c;
    if (!dbg_ok(a.dbg, last, a.rows_o * (D / 4), DBG_LOAD) || !dbg_ok(a.dbg, e, n, DBG_STORE)) return;
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
    cudaError_t e;
    if (a.fast) {
        e = fast::launch_bwd(a, dev, stream);
    } else {
        e = launch_bwd_state(a, dev, stream);
        if (e != cudaSuccess) return e;
        const long long units = (long long)a.slots * a.HV;
        if (units == 0) return cudaSuccess;
        static volatile int done[kMaxDev];
        e = smem_limit_once(kda_chunk_bwd_kernel<T16>, (int)sizeof(Smem), dev, done);
        if (e != cudaSuccess) return e;
        kda_chunk_bwd_kernel<T16><<<units < kSMs ? (unsigned)units : kSMs, kThreads, sizeof(Smem),
                                    stream>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || !a.dq_hv || a.slots == 0) return e;
    const size_t n = 2 * (a.rows_o / (a.HV / a.H)) * (D / 4);
    return launch_early(kda_chunk_bwd_heads_kernel<T16>, (unsigned)((n + 255) / 256), 256, 0, stream,
                        a);
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
