// Backward of the gated delta-rule recurrence for BF16 training, second pass (see kda_fast.cuh,
// and kda_chunk_bwd.cu for the mathematics): dq, dk, dgate and dbeta of every 64-token slot of
// every head at once.  Eight warps own 16 dk channels each; S and its gradient, e, Y and do are
// FP16 operands with a power of two each: one for a warp's rows of S (and of dS), one for a
// step of e, Y and do.  The pairs inside a step carry 2^-g without a bound and stay in three
// BF16 products.
//
// A persistent CTA a SM takes one slot after the other (a slot's operands fill its shared
// memory).  Of a slot's 28 thousand cycles R takes 7, F 9, loads 5, preparing operands 3.5 and the
// pairs' products 1; no unit is saturated: shared-memory pipe 63%, issue slots 40%, tensor cores
// 26%.  Each warp's 16 rows read all of e, Y and do from shared memory.  Sixteen warps, R and F on
// eight each, took longer (860 us).  B=8 T=4096 H=16: 775 us for 8192 slots, 2.4 TB/s.
#include "kda_fast.cuh"
#include "kda_ops.h"

namespace kda {
namespace fast {

cudaError_t launch_bwd_state(const ChunkBwdArgs &a, int dev, cudaStream_t stream);

namespace {

using chunk::cp16z;
using chunk::ldsm4;
using chunk::ldsm4t;
using chunk::mma3;
using chunk::movm_t;
using chunk::mul2;
using chunk::pack_bf16;
using chunk::split2;
using tc::smem_u32;

constexpr int kThreads = 256;
constexpr int QS = D + 8;  // row strides in shared memory: the fragment reads (8 channels of
constexpr int GS = D + 4;  // every second token) fall into different banks

struct __align__(128) Smem {
    // FP16 blocks of 8 tokens by 8 dv, [token / 8][dv / 8]; of e and Y the rows are dv, of do tokens
    char e[kRowsBytes], y[kRowsBytes], dout[kRowsBytes];
    uint16_t q[BT][QS], k[BT][QS];
    float g[BT][GS];                    // cumulative inside each 16-token step
    float beta[BT], diag[BT];           // diag: do_t.e_t
    char g1[4][2 * kTile], g2[4][2 * kTile];  // BF16 hi, lo of each step, zero from the diagonal on
    float col[4][8][kThreads];          // dk_col from R to F, each thread's own
    uint4 state[8][kThreads];           // a saved state on its way, each thread's own part
    char out[3][kThreads / 32][512];    // a warp's dq, dk, dgate of a step on their way out
    uint32_t omax[4];                   // largest |do| of a step
};

__device__ __forceinline__ uint32_t block_at(uint32_t base, int tb, int db, int lane) {
    return base + (uint32_t)((tb * 16 + db) * 128 + (lane & 7) * 16);
}

// A thread's elements of a step: channels gr, gr + 8 (i) of its warp's 16, tokens tc2, tc2 + 1,
// 8 + tc2, 9 + tc2 (p): as left operands, the fragments' words are (i, p) = (0, 01), (1, 01),
// (0, 23), (1, 23).
struct Elems {
    float v[2][4];
};
__device__ __forceinline__ int token_of(int p, int tc2) { return tc2 + (p & 1) + (p >> 1) * 8; }
__device__ __forceinline__ void split_elems(const Elems &x, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(x.v[0][0], x.v[0][1], hi[0], lo[0]);
    split2(x.v[1][0], x.v[1][1], hi[1], lo[1]);
    split2(x.v[0][2], x.v[0][3], hi[2], lo[2]);
    split2(x.v[1][2], x.v[1][3], hi[3], lo[3]);
}
__device__ __forceinline__ void pack_elems(const Elems &x, float f, uint32_t (&a)[4]) {
    a[0] = pack_f16(x.v[0][0] * f, x.v[0][1] * f);
    a[1] = pack_f16(x.v[1][0] * f, x.v[1][1] * f);
    a[2] = pack_f16(x.v[0][2] * f, x.v[0][3] * f);
    a[3] = pack_f16(x.v[1][2] * f, x.v[1][3] * f);
}
__device__ __forceinline__ Elems load_elems(const uint16_t (*rows)[QS], int c0, int lane) {
    uint32_t r[4];
    ldsm4t(r, smem_u32(&rows[(lane & 7) + ((lane >> 4) & 1) * 8][c0 + ((lane >> 3) & 1) * 8]));
    Elems x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf2(r[i]);
        x.v[i & 1][(i >> 1) * 2] = f.x;
        x.v[i & 1][(i >> 1) * 2 + 1] = f.y;
    }
    return x;
}

__device__ __forceinline__ void scale_rows(float (&S)[16][4], float d0, float d1) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float2 u = mul2(make_float2(S[j][0], S[j][1]), make_float2(d0, d0));
        const float2 w = mul2(make_float2(S[j][2], S[j][3]), make_float2(d1, d1));
        S[j][0] = u.x; S[j][1] = u.y; S[j][2] = w.x; S[j][3] = w.y;
    }
}
__device__ __forceinline__ void operand(const float (&S)[16][4], int kk, uint32_t (&a)[4]) {
    const float(&x)[4] = S[2 * kk], (&y)[4] = S[2 * kk + 1];
    a[0] = pack_f16(x[0], x[1]);
    a[1] = pack_f16(x[2], x[3]);
    a[2] = pack_f16(y[0], y[1]);
    a[3] = pack_f16(y[2], y[3]);
}

// A step's pairs where k 2^-g would leave FP32's range: one exp2 per (r, s, channel), the
// thread's tokens as rows (dq, dk_row; add to what is there) or as columns (dk_col).
__device__ __noinline__ void pairs_strong(Smem &sm, int j, int c0, int lane, float scale,
                                          bool columns, Elems &x, Elems &y) {
    auto tile = [](const char *t, int r, int s) {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(t) + r * C + s;
        return bf1(h[0]) + bf1(h[C * C]);
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
                    const float kb = sm.beta[j * C + s] * bf1(sm.k[j * C + s][ch]) *
                                     ex2(gt - sm.g[j * C + s][ch]);
                    u += tile(sm.g1[j], t, s) * kb;
                    w += tile(sm.g2[j], t, s) * kb;
                }
                x.v[i][p] += scale * u;
                y.v[i][p] -= sm.beta[j * C + t] * w;
            } else {
                for (int r = t + 1; r < C; ++r) {
                    const float q = scale * bf1(sm.q[j * C + r][ch]);
                    const float k = sm.beta[j * C + r] * bf1(sm.k[j * C + r][ch]);
                    u += (tile(sm.g1[j], r, t) * q - tile(sm.g2[j], r, t) * k) *
                         ex2(sm.g[j * C + r][ch] - gt);
                }
                x.v[i][p] += sm.beta[j * C + t] * u;
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1) kda_fast_bwd_kernel(const ChunkBwdArgs a) {
    extern __shared__ __align__(128) char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, warp = chunk::warp_index(), lane = tid & 31;
    const int gr = lane >> 2, tc2 = (lane & 3) * 2, m = lane >> 3;
    const int c0 = warp * 16;  // this warp's channels
    const uint32_t se = smem_u32(sm.e), sy = smem_u32(sm.y), so = smem_u32(sm.dout);
    // lanes' offsets of a [16][16] tile as right operand: rows as columns, or rows summed over
    const uint32_t tn = chunk::tile_lane(lane);
    const uint32_t tt = (uint32_t)(((lane & 7) + ((lane >> 3) & 1) * 8) * 32 + (lane >> 4) * 16);
    // a unit's saved blocks take 57 KB, so that their number is far below 2^31
    const unsigned units = (unsigned)a.slots * a.HV;

    // a thread's words of a saved state, asked for long before they are used
    auto fetch_state = [&](const char *base, unsigned u) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
            cp_async16(&sm.state[t][tid], base + (size_t)u * kCkptBytes + (t * kThreads + tid) * 16);
        cp_async_commit();
    };

    chunk::Where next = chunk::locate(a, blockIdx.x);
    fetch_state(a.dckpt, blockIdx.x);
    for (unsigned u = blockIdx.x; u < units; u += gridDim.x) {
        const long long row0 = next.row0;
        const unsigned after = u + gridDim.x;
        const int rows = next.rows, h = next.h, hv = next.hv;
        if (rows <= 0) {  // no tokens here (the same for every thread)
            cp_async_wait_all();
            if (after < units) {
                next = chunk::locate(a, after);
                fetch_state(a.dckpt, after);
            }
            continue;
        }
        const size_t su = (size_t)u;

        // ---- loads
        if (tid < 4) sm.omax[tid] = 0u;
        // do: eight rows at a time, so that a lane's piece of its FP16 block falls into banks of
        // its own
        const int o_row = (lane & 7) + (warp >> 2) * 8, o_col = (warp & 3) * 4 + (lane >> 3);
        uint4 dor[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = 16 * x + o_row;
            dor[x] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows && chunk::token_ok(a, row0 + r))
                dor[x] = *reinterpret_cast<const uint4 *>(
                    (const uint16_t *)a.dout + ((size_t)(row0 + r) * a.HV + hv) * D + o_col * 8);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = (tid >> 4) + 16 * x, c = tid & 15;
            const bool ok = r < rows && chunk::token_ok(a, row0 + r);
            const size_t tok = (size_t)(row0 + (ok ? r : 0));
            cp16z(smem_u32(&sm.q[r][c * 8]), (const uint16_t *)a.q + (tok * a.H + h) * D + c * 8, ok);
            cp16z(smem_u32(&sm.k[r][c * 8]), (const uint16_t *)a.k + (tok * a.H + h) * D + c * 8, ok);
            const size_t iv = (tok * a.HV + hv) * D;
            cp16z(smem_u32(&sm.g[r][c * 4]), a.gate + iv + c * 4, ok);
            cp16z(smem_u32(&sm.g[r][64 + c * 4]), a.gate + iv + 64 + c * 4, ok);
        }
        cp_async_commit();
        // e and Y: a warp has tile `warp` of the four steps; lane 8j + t knows the scale of
        // step j, tile t
        uint4 er[4], yr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            er[j] = reinterpret_cast<const uint4 *>(a.e + su * kRowsBytes)[(j * 8 + warp) * 32 + lane];
            yr[j] = reinterpret_cast<const uint4 *>(a.y + su * kRowsBytes)[(j * 8 + warp) * 32 + lane];
        }
        const float es = a.scales[su * kScales + 8 + lane], ys = a.dscales[su * kScales + 8 + lane];
        const float cs = a.scales[su * kScales + (lane & 7)];
        const float ds = a.dscales[su * kScales + (lane & 7)];
        if (tid < BT)
            sm.beta[tid] = tid < rows && chunk::token_ok(a, row0 + tid) ? a.beta[(size_t)(row0 + tid) * a.HV + hv] : 0.f;
        // a warp's 16 rows of a saved state: tile t of 16 dv columns is the word pair w of its
        // blocks; brought to the common scale `c` of the eight tiles
        float S[16][4];  // rows dk c0 + gr, + 8; columns dv 8j + tc2, + 1
        auto load_state = [&](float scales, float c, int t, float (&l)[4], float (&r)[4]) {
            const uint4 w = sm.state[t][tid];
            const float f = c * inverse_of(__shfl_sync(0xffffffffu, scales, t));
            auto put = [&](uint32_t x, float &first, float &second) {
                const uint32_t y = movm_t(x);
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&y));
                first = v.x * f;
                second = v.y * f;
            };
            put(w.x, l[0], l[1]);
            put(w.y, r[0], r[1]);
            put(w.z, l[2], l[3]);
            put(w.w, r[2], r[3]);
        };
        auto least8 = [&](float x) {
#pragma unroll
            for (int off = 1; off < 8; off <<= 1)
                x = fminf(x, __shfl_xor_sync(0xffffffffu, x, off));
            return x;
        };
        const float ce = least8(es), cy = least8(ys);  // of the lane's step (lane / 8)
        const float c_state = least8(cs), d_state = least8(ds);
        // blocks of e and Y at the step's common scale
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            auto rescaled = [&](const uint4 &w, float own, float common, char *to) {
                const float f = __shfl_sync(0xffffffffu, common, 8 * j) *
                                inverse_of(__shfl_sync(0xffffffffu, own, 8 * j + warp));
                const __half2 hf = __float2half2_rn(f);
                auto one = [&](uint32_t x) {
                    const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x), hf);
                    return *reinterpret_cast<const uint32_t *>(&y);
                };
                char *p = to + (2 * j * 16 + 2 * warp) * 128 + lane * 4;
                *reinterpret_cast<uint32_t *>(p) = one(w.x);
                *reinterpret_cast<uint32_t *>(p + 128) = one(w.y);
                *reinterpret_cast<uint32_t *>(p + 16 * 128) = one(w.z);
                *reinterpret_cast<uint32_t *>(p + 17 * 128) = one(w.w);
            };
            rescaled(er[j], es, ce, sm.e);
            rescaled(yr[j], ys, cy, sm.y);
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // rows 16x ..: step x
            uint32_t mx = __vmaxu2(__vmaxu2(dor[x].x & 0x7fff7fffu, dor[x].y & 0x7fff7fffu),
                                   __vmaxu2(dor[x].z & 0x7fff7fffu, dor[x].w & 0x7fff7fffu));
            mx = __reduce_max_sync(0xffffffffu, max(mx << 16, mx & 0xffff0000u));
            if (lane == 0) atomicMax(&sm.omax[x], mx);
        }
        cp_async_wait_all();
        __syncthreads();
        float co[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            co[x] = scale_for(fmaxf(__uint_as_float(sm.omax[x]), 1e-30f), kTop);
            auto one = [&](uint32_t v) {
                const float2 f = bf2(v);
                return pack_f16(f.x * co[x], f.y * co[x]);
            };
            *reinterpret_cast<uint4 *>(
                sm.dout + ((2 * x + (warp >> 2)) * 16 + o_col) * 128 + (lane & 7) * 16) =
                make_uint4(one(dor[x].x), one(dor[x].y), one(dor[x].z), one(dor[x].w));
        }
        // ---- cumulative gate inside each step
        for (int i = tid; i < 4 * D; i += kThreads) {
            const int ch = i & (D - 1), j = i / D;
            float acc = 0.f;
#pragma unroll
            for (int r = 0; r < C; ++r) {
                acc += chunk::floor_gate(sm.g[j * C + r][ch]);
                sm.g[j * C + r][ch] = acc;
            }
        }
        // scales of a step, for every lane
        auto of_step = [&](float x, int j) { return __shfl_sync(0xffffffffu, x, 8 * j); };
        // ---- scales of the warp's rows of S and dS: room for what the four steps add to them
        float cS, cD;
        {
            uint32_t qb = 0u, kb = 0u;
#pragma unroll
            for (int x = 0; x < 4; ++x) {  // 16 tokens a time, two pieces of a row
                const int r = 16 * x + (lane >> 1), c = c0 + (lane & 1) * 8;
                const uint4 q = *reinterpret_cast<const uint4 *>(&sm.q[r][c]);
                const uint4 k = *reinterpret_cast<const uint4 *>(&sm.k[r][c]);
                auto most = [](uint32_t m, const uint4 &v) {
                    m = __vmaxu2(__vmaxu2(m, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
                    return __vmaxu2(__vmaxu2(m, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
                };
                qb = most(qb, q);
                kb = most(kb, k);
            }
            auto over_warp = [](uint32_t m) {
                return __uint_as_float(
                    __reduce_max_sync(0xffffffffu, max(m << 16, m & 0xffff0000u)));
            };
            const float qm = fabsf(a.scale) * over_warp(qb);
            const float km = over_warp(kb) *
                             warp_max(fmaxf(fabsf(sm.beta[lane]), fabsf(sm.beta[32 + lane])));
            float e_sum = 0.f, d_sum = 0.f;  // 2^14 of the operands' own scales
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                e_sum += inverse_of(of_step(ce, j));
                d_sum += qm * inverse_of(co[j]) + km * inverse_of(of_step(cy, j));
            }
            const float top = 1.f / (C * 16384.f);  // one step: 16 tokens of operands below 2^14
            auto room = [&](float c, float sum) {
                const float lim = scale_for(fmaxf(sum / top, 1e-20f), kTop);
                return fminf(c, lim);
            };
            cS = room(c_state, km * e_sum);
            cD = room(d_state, d_sum);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) load_state(ds, cD, t, S[2 * t], S[2 * t + 1]);
        fetch_state(a.ckpt, u);
        __syncthreads();
        // ---- the pairs' products
        {
            const int j = warp & 3;  // warps 0-3: do.e, warps 4-7: Y.e of step j
            float c[2][4] = {};
#pragma unroll 4
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t af[4], bf[4];
                if (warp < 4)
                    ldsm4(af, block_at(so, 2 * j + (m & 1), 2 * kk + (m >> 1), lane));
                else
                    ldsm4t(af, block_at(sy, 2 * j + (m & 1), 2 * kk + (m >> 1), lane));
                ldsm4t(bf, block_at(se, 2 * j + (m >> 1), 2 * kk + (m & 1), lane));
                mma_f16(c[0], af, bf[0], bf[1]);
                mma_f16(c[1], af, bf[2], bf[3]);
            }
            const float cj = j == 0 ? co[0] : j == 1 ? co[1] : j == 2 ? co[2] : co[3];
            const float f1 = inverse_of(of_step(ce, j));
            const float f2 = inverse_of(warp < 4 ? cj : of_step(cy, j));
            char *to = warp < 4 ? sm.g1[j] : sm.g2[j];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; p += 2) {
                    const int r = gr + p * 4, s = 8 * i + tc2, t = j * C + r;
                    const float x = c[i][p] * f1 * f2, y = c[i][p + 1] * f1 * f2;
                    uint32_t hi, lo;
                    split2(s < r ? x : 0.f, s + 1 < r ? y : 0.f, hi, lo);
                    *reinterpret_cast<uint32_t *>(to + (r * C + s) * 2) = hi;
                    *reinterpret_cast<uint32_t *>(to + kTile + (r * C + s) * 2) = lo;
                    if (r == s || r == s + 1) {
                        const float d = r == s ? x : y;
                        if (warp < 4)
                            sm.diag[t] = d;
                        else if (t < rows && chunk::token_ok(a, row0 + t))
                            chunk::put_dbeta(a, (size_t)(row0 + t) * a.HV + hv, d,
                                      (uint16_t)(pack_bf16(d, 0.f) & 0xffffu));
                    }
                }
        }
        __syncthreads();

        // the next unit's inputs are asked into L2 while the loads' queue is empty
        if (after < units) {
            next = chunk::locate(a, after);
            const size_t nu = (size_t)after;
            if (tid == 0) {
                tc::prefetch_l2(a.e + nu * kRowsBytes, (uint32_t)kRowsBytes);
                tc::prefetch_l2(a.y + nu * kRowsBytes, (uint32_t)kRowsBytes);
                tc::prefetch_l2(a.ckpt + nu * kCkptBytes, (uint32_t)kCkptBytes);
            }
            chunk::prefetch_rows(a, next, tid, kThreads);
        }
        // ---- R
#pragma unroll 1
        for (int j = 3; j >= 0; --j) {
            const float cj = j == 0 ? co[0] : j == 1 ? co[1] : j == 2 ? co[2] : co[3];
            const float ej = of_step(ce, j), yj = of_step(cy, j);
            float cd[2][4] = {}, cd2[2][4] = {};  // two chains a tile
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t af[4], bf[4];
                ldsm4t(bf, block_at(se, 2 * j + (m >> 1), 2 * kk + (m & 1), lane));
                operand(S, kk, af);
                mma_f16(kk & 1 ? cd2[0] : cd[0], af, bf[0], bf[1]);
                mma_f16(kk & 1 ? cd2[1] : cd[1], af, bf[2], bf[3]);
            }
            const Elems q = load_elems(&sm.q[j * C], c0, lane);
            const Elems k = load_elems(&sm.k[j * C], c0, lane);
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
            const bool strong = __any_sync(0xffffffffu, big > 96.f);
            const float d0 = ex2(gl[0]), d1 = ex2(gl[1]);
            const float f = inverse_of(cD) * inverse_of(ej);
            const float f0 = strong ? f : f * d0, f1 = strong ? f : f * d1;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                cd[x][0] = (cd[x][0] + cd2[x][0]) * f0;
                cd[x][1] = (cd[x][1] + cd2[x][1]) * f0;
                cd[x][2] = (cd[x][2] + cd2[x][2]) * f1;
                cd[x][3] = (cd[x][3] + cd2[x][3]) * f1;
            }
            if (!strong) {
                uint32_t ah[4], al[4], wh[4], wl[4], bh[4], bl[4], ch[4], cl[4];
                split_elems(qw, ah, al);
                split_elems(kw, wh, wl);
                ldsm4t(bh, smem_u32(sm.g1[j]) + tt);
                ldsm4t(bl, smem_u32(sm.g1[j]) + kTile + tt);
                ldsm4t(ch, smem_u32(sm.g2[j]) + tt);
                ldsm4t(cl, smem_u32(sm.g2[j]) + kTile + tt);
                mma3(cd[0], cd[1], ah, al, bh, bl);
                mma3(cd[0], cd[1], wh, wl, ch, cl);
            }
            Elems col;
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
                pairs_strong(sm, j, c0, lane, a.scale, true, x, x);
                col = x;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) sm.col[j][4 * i + p][tid] = col.v[i][p];
            // dS <- 2^g_l dS' + qw^T do - (beta kw)^T Y
            uint32_t qf[4], kf[4];
            pack_elems(qw, cD * inverse_of(cj), qf);
            pack_elems(kw, cD * inverse_of(yj), kf);
            scale_rows(S, d0, d1);
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) {
                uint32_t bf[4], yf[4];
                ldsm4t(bf, block_at(so, 2 * j + (m & 1), 2 * jj + (m >> 1), lane));
                ldsm4(yf, block_at(sy, 2 * j + (m & 1), 2 * jj + (m >> 1), lane));
                mma_f16(S[2 * jj], qf, bf[0], bf[1]);
                mma_f16(S[2 * jj + 1], qf, bf[2], bf[3]);
                mma_f16(S[2 * jj], kf, yf[0], yf[1]);
                mma_f16(S[2 * jj + 1], kf, yf[2], yf[3]);
            }
        }
        // ---- the state at the slot's start, and sum_dv S dS there
        float carry[2] = {0.f, 0.f};
        cp_async_wait_all();
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float x[2][4];
            load_state(cs, cS, t, x[0], x[1]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float(&s)[4] = S[2 * t + y];
                carry[0] += s[0] * x[y][0] + s[1] * x[y][1];
                carry[1] += s[2] * x[y][2] + s[3] * x[y][3];
#pragma unroll
                for (int p = 0; p < 4; ++p) s[p] = x[y][p];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            carry[i] *= inverse_of(cS) * inverse_of(cD);
            carry[i] += __shfl_xor_sync(0xffffffffu, carry[i], 1);
            carry[i] += __shfl_xor_sync(0xffffffffu, carry[i], 2);
        }
        if (after < units) fetch_state(a.dckpt, after);
        // ---- F, and the outputs
        const size_t orow = (size_t)a.HV * D;
        const size_t out_at = (size_t)row0 * orow + (size_t)hv * D + c0;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const float cj = j == 0 ? co[0] : j == 1 ? co[1] : j == 2 ? co[2] : co[3];
            const float ej = of_step(ce, j), yj = of_step(cy, j);
            float cq[2][4] = {}, cyy[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t af[4], bf[4], yf[4];
                ldsm4(bf, block_at(so, 2 * j + (m >> 1), 2 * kk + (m & 1), lane));
                ldsm4t(yf, block_at(sy, 2 * j + (m >> 1), 2 * kk + (m & 1), lane));
                operand(S, kk, af);
                mma_f16(cq[0], af, bf[0], bf[1]);
                mma_f16(cq[1], af, bf[2], bf[3]);
                mma_f16(cyy[0], af, yf[0], yf[1]);
                mma_f16(cyy[1], af, yf[2], yf[3]);
            }
            const Elems q = load_elems(&sm.q[j * C], c0, lane);
            const Elems k = load_elems(&sm.k[j * C], c0, lane);
            Elems kb, kd, g;
            float gl[2], big = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                gl[i] = sm.g[j * C + C - 1][c0 + gr + 8 * i];
                big = fmaxf(big, -gl[i]);
            }
            const bool strong = __any_sync(0xffffffffu, big > 96.f);
            // the pairs' factors from the middle of the step's decay on: 2^-g itself reaches 2^96,
            // beside which large values would leave FP32's range
            const float mid[2] = {strong ? 0.f : 0.5f * gl[0], strong ? 0.f : 0.5f * gl[1]};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int t = j * C + token_of(p, tc2);
                    g.v[i][p] = sm.g[t][c0 + gr + 8 * i];
                    const float x = sm.beta[t] * k.v[i][p];
                    kb.v[i][p] = x * ex2(mid[i] - g.v[i][p]);
                    kd.v[i][p] = x * ex2(gl[i] - g.v[i][p]);
                }
            const float m0 = ex2(mid[0]), m1 = ex2(mid[1]);
            const float fq = inverse_of(cS) * inverse_of(cj), fy = inverse_of(cS) * inverse_of(yj);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    cq[x][p] *= fq * (p < 2 ? m0 : m1);
                    cyy[x][p] *= fy * (p < 2 ? m0 : m1);
                }
            if (!strong) {
                uint32_t ah[4], al[4], bh[4], bl[4], ch[4], cl[4];
                split_elems(kb, ah, al);
                ldsm4(bh, smem_u32(sm.g1[j]) + tn);
                ldsm4(bl, smem_u32(sm.g1[j]) + kTile + tn);
                ldsm4(ch, smem_u32(sm.g2[j]) + tn);
                ldsm4(cl, smem_u32(sm.g2[j]) + kTile + tn);
                chunk::mma3x2<true>(cq[0], cq[1], cyy[0], cyy[1], ah, al, bh, bl, ah, al, ch, cl);
            }
            if (j < 3) {  // S <- 2^g_l S + (beta k 2^(g_l - g))^T e
                uint32_t kf[4];
                pack_elems(kd, cS * inverse_of(ej), kf);
                scale_rows(S, ex2(gl[0]), ex2(gl[1]));
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
                    uint32_t bf[4];
                    ldsm4(bf, block_at(se, 2 * j + (m & 1), 2 * jj + (m >> 1), lane));
                    mma_f16(S[2 * jj], kf, bf[0], bf[1]);
                    mma_f16(S[2 * jj + 1], kf, bf[2], bf[3]);
                }
            }
            Elems dq, dk;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float up = ex2(g.v[i][p] - mid[i]);
                    dq.v[i][p] = a.scale * up * cq[p >> 1][2 * i + (p & 1)];
                    dk.v[i][p] = -sm.beta[j * C + token_of(p, tc2)] * up *
                                 cyy[p >> 1][2 * i + (p & 1)];
                }
            if (strong) {
                Elems x = dq, y = dk;
                pairs_strong(sm, j, c0, lane, a.scale, false, x, y);
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
                    w[y] = pack_bf16(x.v[y & 1][y & 2], x.v[y & 1][(y & 2) + 1]);
                chunk::store_out(sm.out[which][warp], w,
                                    (char *)((uint16_t *)out + out_at + (size_t)j * C * orow),
                                    orow * 2, rows - j * C, (char *)out, a.rows_o * D * 2, a.dbg,
                                    lane);
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

}  // namespace

// The slots' gradients; dq and dk of grouped heads are still to be summed when dq_hv is set.
cudaError_t launch_bwd(const ChunkBwdArgs &a, int dev, cudaStream_t stream) {
    cudaError_t e = launch_bwd_state(a, dev, stream);
    if (e != cudaSuccess) return e;
    const long long units = (long long)a.slots * a.HV;
    if (units == 0) return cudaSuccess;
    static volatile int done[kMaxDev];
    e = smem_limit_once(kda_fast_bwd_kernel, (int)sizeof(Smem), dev, done);
    if (e != cudaSuccess) return e;
    kda_fast_bwd_kernel<<<units < kSMs ? (unsigned)units : kSMs, kThreads, sizeof(Smem), stream>>>(
        a);
    return cudaGetLastError();
}

}  // namespace fast
}  // namespace kda
