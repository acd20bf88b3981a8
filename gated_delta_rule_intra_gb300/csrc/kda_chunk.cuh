// Shared parts of the gated delta-rule recurrence kernels (forward and backward).
//
// Per value head the state S is [128 dk, 128 dv] in FP32.  A token decays it per channel,
// S~ = diag(2^gate) S, and corrects it towards its value: e = v - S~^T k,
// S' = S~ + beta k e^T, o = scale S'^T q.  The kernels walk a sequence in steps of C = 16
// tokens.  With g the inclusive cumsum of the gate inside the step and g_l its last row,
//   kw = k 2^g,  qw = scale q 2^g,  kd = k 2^(g_l - g),
//   M[r,s] = sum_d k_r k_s 2^(g_r - g_s) (s < r),  P[r,s] = scale sum_d q_r k_s 2^(..) (s <= r)
//   e = T2 (v - kw S) with T2 = (I + M diag(beta))^-1,   n = beta e,
//   o = qw S + P n,   S' = diag(2^g_l) S + kd^T n
// and backwards, with T = (I + diag(beta) M)^-1,
//   dn = P^T do + kd dS',  Y = T^T dn,  dv = beta Y,
//   dS = diag(2^g_l) dS' + qw^T do - kw^T (beta Y).
// Every exponent is <= 0 for gates <= 0.  e, n and Y do not depend on where steps begin.
//
// The state never leaves the registers: each consumer warp owns 16 of the 128 dv columns of
// S as the accumulators of S^T [16 dv, 128 dk], which are also the fragments of the next
// product's left operand, so the chain S -> kw S -> e -> S' has no shared-memory round trip
// and no exchange between warps.  That is why these kernels use mma.sync: a step's products
// have 16 or 32 columns, and a tensor-memory accumulator would have to come back through the
// registers (to be rounded to operands) three times a step.
//
// Precision: products of FP32 values are taken as three BF16 products with FP32 sums, x being
// hi + lo with hi = bf16(x), lo = bf16(x - hi): 16 bits of x are kept (2^-17 relative), the
// dropped lo * lo is below 2^-16 of the product, and BF16 keeps FP32's range, which a state
// that a user may scale freely needs.  A TF32 operand would keep 11 bits at half the rate.
#pragma once

#include "kda_ops.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace chunk {

constexpr int C = 16;            // tokens a step
constexpr int D = KD;            // channels of q and k, and of v
constexpr int kPrepThreads = 256;
constexpr int kPlane = C * D * 2;      // bytes of a BF16 [16][128] operand plane
constexpr int kTile = C * C * 2;       // bytes of a BF16 [16][16] tile
constexpr size_t kCkptBytes = 2 * D * D * 2;  // a state checkpoint: hi and lo planes
constexpr size_t kRowPlane = BT * D * 2;      // one BF16 plane of 64 rows of dv
constexpr size_t kRowsBytes = 2 * kRowPlane;  // e or Y of 64 tokens: hi and lo planes
constexpr size_t kTilesBytes = 4 * kTile;     // T hi, T lo, P hi, P lo of a step

// Gates below this are taken as this: 2^-160 is 0 in FP32 either way, and differences of the
// cumulative gate stay finite for gates of the type's lowest value or -infinity.  NaN stays.
__device__ __forceinline__ float floor_gate(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-160.f));
    return y;
}

using kda::add2;
using kda::fma2;
using kda::mul2;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// (x, y) as two BF16 pairs: hi = bf16(.), lo = bf16(. - hi)
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    const float2 d = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)),
                          make_float2(-1.f, -1.f), make_float2(x, y));
    lo = pack_bf16(d.x, d.y);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// Transpose of an 8x8 matrix of 16-bit values held in fragment order by a warp.
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int n) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// bar_sync() that also tells whether any of its threads passed true.
__device__ __forceinline__ bool bar_or(int id, int n, bool x) {
    int r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %3, 0;\nbarrier.cta.red.or.pred q, %1, %2, p;\n"
                 "selp.b32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"(id), "r"(n), "r"((int)x)
                 : "memory");
    return r != 0;
}
// cp.async of 16 (or 4) bytes, zeros when !ok.
__device__ __forceinline__ void cp16z(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp4z(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 4 : 0)
                 : "memory");
}
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of the 16-byte chunk c of row r in a swizzled [16][128] BF16 plane: the eight
// rows that one ldmatrix phase reads fall into different banks.
__device__ __forceinline__ uint32_t plane_off(int r, int c) {
    return (uint32_t)(r * 256 + ((c ^ (r & 7)) << 4));
}

// A value that is the same in all lanes, said so that the compiler knows it too: branches on
// it are then warp-uniform.  (Behind a branch that might diverge every ldmatrix, mma and shuffle
// waits for the whole warp and nothing is scheduled across it: two to four times the time.)
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int warp_index() { return uniform((int)(threadIdx.x >> 5)); }

// A sequence: its rows in the [rows, heads, 128] tensors and its slots of 64 tokens.
struct Seq {
    long long row0;  // first token
    int len;         // tokens
    int slot0;       // first 64-token slot in the checkpoint buffers
};

// Sequence n of the launch.  Fixed length: n = batch index.  Variable length: the tokens
// [cu[n], cu[n+1]) clamped to the packed length, slots from cu[n] / 64 + n on (no two
// sequences' slots meet, and T / 64 + num_seqs + 1 slots cover every input).
__device__ __forceinline__ int2 range_of(int n, int T, const int *cu) {
    int a = cu[n], b = cu[n + 1];
    a = a < 0 ? 0 : a > T ? T : a;
    b = b < a ? a : b > T ? T : b;
    return make_int2(a, b);
}
// The same n in all lanes of the warp.
__device__ __forceinline__ Seq seq_of(int n, int T, const int *cu) {
    Seq s;
    if (cu) {
        const int2 x = range_of(n, T, cu);
        s.row0 = uniform(x.x);
        s.len = uniform(x.y - x.x);
        s.slot0 = uniform(x.x / BT + n);
    } else {
        s.row0 = (long long)n * T;
        s.len = T;
        s.slot0 = n * ((T + BT - 1) / BT);
    }
    return s;
}

__device__ __forceinline__ void prefetch_line(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The tokens of unit u (a slot of a value head); rows <= 0 where there are none.
struct Where {
    long long row0;
    int rows, h, hv;
};
__device__ __forceinline__ Where locate(const ChunkBwdArgs &a, unsigned u) {
    Where w;
    const int slot = (int)(u / (unsigned)a.HV);
    w.hv = (int)u - slot * a.HV;
    w.h = w.hv / (a.HV / a.H);
    int n;  // the slot's sequence
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
    const int t0 = (slot - sq.slot0) * BT;
    w.row0 = sq.row0 + t0;
    w.rows = t0 < 0 ? 0 : min(BT, sq.len - t0);
    return w;
}

// The debug build's checks: a token of the inputs, and a head's state from element `at` on (its last
// 16 rows lie behind that in any split).
template <class Args> __device__ __forceinline__ bool token_ok(const Args &a, long long token) {
    return dbg_ok(a.dbg, (size_t)token, a.rows_o / a.HV, DBG_LOAD);
}
template <class Args>
__device__ __forceinline__ bool state_ok(const Args &a, const void *p, size_t at, unsigned bit) {
    return !p || dbg_ok(a.dbg, at / (D * D) * (D * D) + D * D - 1, a.states, bit);
}

// An element of dbeta: FP32, or what it is in 16 bits.
__device__ __forceinline__ void put_dbeta(const ChunkBwdArgs &a, size_t at, float x, uint16_t x16) {
    if (a.gates32)
        ((float *)a.dbeta)[at] = x;
    else
        ((uint16_t *)a.dbeta)[at] = x16;
}

// Asks a unit's rows of q, k and do (two lines each) and of the gate (four) into L2.
__device__ __forceinline__ void prefetch_rows(const ChunkBwdArgs &a, const Where &w, int tid,
                                              int threads) {
    for (int x = tid; x < 10 * BT; x += threads) {
        const int r = x / 10, l = x - 10 * r;
        if (r >= w.rows) break;
        const size_t tok = (size_t)(w.row0 + r);
        const size_t iq = (tok * a.H + w.h) * D, iv = (tok * a.HV + w.hv) * D;
        const char *p = l < 2   ? (const char *)((const uint16_t *)a.q + iq)
                        : l < 4 ? (const char *)((const uint16_t *)a.k + iq)
                        : l < 6 ? (const char *)((const uint16_t *)a.dout + iv)
                                : (const char *)(a.gate + iv);
        prefetch_line(p + (l < 6 ? l & 1 : l - 6) * 128);
    }
}

// The sequence that is `rank`-th in length, the longest first: a batch of ragged sequences has
// its longest walks begun at once and the short ones fill in behind them.  Sequences of one
// length, and batches too large to be worth ranking, keep their order.  All threads call it.
constexpr int kRanked = 128;
__device__ __forceinline__ int by_length(int rank, int num_seqs, int T, const int *cu) {
    if (!cu || num_seqs > kRanked) return rank;
    __shared__ int len[kRanked], found;
    const int i = threadIdx.x;
    if (i < num_seqs) {
        const int2 x = range_of(i, T, cu);
        len[i] = x.y - x.x;
    }
    __syncthreads();
    if (i < num_seqs) {
        int before = 0;
        for (int j = 0; j < num_seqs; ++j) before += len[j] > len[i] || (len[j] == len[i] && j < i);
        if (before == rank) found = i;
    }
    __syncthreads();
    return uniform(found);
}

// CTAs that a head's 128 dv columns are divided between: the fewest rounds over the SMs.  A
// finer split repeats the preparation, but its step is shorter: a step of the precise forward
// takes 4.8, 3.3 and 2.8 thousand cycles in one, two and four CTAs a head (prefill of T=2048: 304
// us for 128 heads, 204 for 64, 175 for 32).  Of sequences of unknown lengths the longest is
// taken to be four times the average, and the others to fill in behind it (ten prompts of 1 to
// 2609 tokens, 16 heads: 404 us in one CTA a head, 259 in two, 257 in four).  Packed sequences of one
// length lose by that: 1024 tokens of 4 x 16 heads take 182 us where they take 107 unpacked, of 8 x
// 16 heads 215 and 159, of 12 x 16 heads 320 and 311.  BF16 training goes by the same costs (its
// own steps take 3.7 and 2.9 thousand cycles forwards, 3.1, 2.2 and 1.8 backwards).
inline int best_split(int num_seqs, int HV, const int *cu) {
    constexpr int kSplit[3] = {1, 2, 4}, kStep[3] = {47, 33, 27};
    const long long heads = (long long)num_seqs * HV;
    int best = 4;
    double least = 1e300;
    for (int i = 2; i >= 0; --i) {
        const double share = (double)heads * kSplit[i] / kSMs;
        const double cost =
            kStep[i] * (cu ? 4.0 + share : (double)((heads * kSplit[i] + kSMs - 1) / kSMs));
        if (cost < least) {
            least = cost;
            best = kSplit[i];
        }
    }
    return best;
}

// Raw inputs of a step in shared memory.
struct __align__(16) RawStage {
    uint16_t q[C][D];
    uint16_t k[C][D];
    float gate[C][D];
};

// Which warps do what: NW consume, PREP prepare operands (and take the scores), SOLVERS solve the
// steps' triangular systems.  Two consumers have two of the SM's four schedulers to themselves and
// leave the other two to the preparing warps: warps go to the schedulers in turn, and the warps in
// between leave at once.
//
// Registers move from the feeding warps to the consumers, by groups of four warps: both shares
// add up to no more than the kernel is launched with (65,536 over its threads, in eights), which
// ready_once() checks, because a consumer would wait for the rest forever.
template <int NW, int PREP, int SOLVERS> struct Roles {
    static constexpr bool kApart = NW == 2;
    static constexpr int kGroup = kApart ? 4 : NW;  // warps that take registers
    static constexpr int kThreads = kApart ? 640 : 32 * (NW + PREP + SOLVERS);
    static constexpr int kGive = kThreads > 512   ? (NW == 8 ? 64 : 80)
                                 : kThreads == 512 && NW == 4 ? 88 : 112;
    static constexpr int kTake = kThreads > 512 && NW != 8 ? 160 : NW == 8 ? 144 : 248;
    static constexpr int kLaunch = 65536 / kThreads / 8 * 8;
    static_assert(kGroup % 4 == 0 && PREP % 4 == 0 && SOLVERS % 4 == 0, "");
    static_assert(!kApart || (PREP == 8 && SOLVERS == 0), "");
    static_assert(kGroup * 32 * kTake + (kThreads - kGroup * 32) * kGive <= kLaunch * kThreads, "");

    int prep, solver, consumer;  // index, or -1
    bool feeds;                  // prepares or solves (or idles next to those)
    __device__ __forceinline__ explicit Roles(int warp) : prep(-1), solver(-1), consumer(-1) {
        feeds = warp >= kGroup;
        if (!feeds) {
            if (warp < NW) consumer = warp;
        } else if (kApart) {
            if (warp & 2) prep = (warp - kGroup) / 4 * 2 + (warp & 1);
        } else if (warp < kGroup + PREP) {
            prep = warp - kGroup;
        } else {
            solver = warp - kGroup - PREP;
        }
    }
    static __device__ __forceinline__ void give() {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGive));
    }
    static __device__ __forceinline__ void take() {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTake));
    }
};

// A kernel of these roles may be launched: its shared memory is allowed, and it starts with the
// registers that its warps are going to share out.
template <class R, class Kernel>
cudaError_t ready_once(Kernel *kernel, int smem, int dev, volatile int *done) {
    if (dev >= 0 && dev < kMaxDev && done[dev]) return cudaSuccess;
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs != R::kLaunch) return cudaErrorLaunchOutOfResources;
    return smem_limit_once(kernel, smem, dev, done);
}

template <typename T16> __device__ __forceinline__ float2 unpack2(uint32_t x);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}
template <typename T16> __device__ __forceinline__ uint32_t pack2(float x, float y);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
    return pack_bf16(x, y);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
    __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<uint32_t *>(&h);
}

// The six operand planes of a step.
enum { KW_HI = 0, KW_LO, QW_HI, QW_LO, KD_HI, KD_LO, kPlanes };

__device__ __forceinline__ void put_split(char *hi_plane, uint32_t off, float x, float y) {
    uint32_t hi, lo;
    split2(x, y, hi, lo);
    *reinterpret_cast<uint32_t *>(hi_plane + off) = hi;
    *reinterpret_cast<uint32_t *>(hi_plane + kPlane + off) = lo;
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Operand planes of a step from its raw inputs: NT threads, each two channels of C * 64 / NT
// rows.  Writes kw, qw, 2^g_l and the key plane: k 2^(g_l - g), or with FROM_START k 2^-g,
// which may grow without bound.  Returns whether the latter will not do: a key grew past 2^96 or is
// NaN, or a channel lost more than 2^-100 (2^-g leaves FP32's range soon after, and a key of
// zero times infinity would be NaN).
template <typename T16, int NT, bool FROM_START>
__device__ __forceinline__ bool prep_planes(const RawStage &raw, char *planes, float *decay,
                                            float scale, int tid) {
    constexpr int kRows = C * 64 / NT;
    const int c2 = tid & 63, r0 = (tid >> 6) * kRows;
    auto gate = [&](int r) {
        const float2 x = *reinterpret_cast<const float2 *>(&raw.gate[r][2 * c2]);
        return make_float2(floor_gate(x.x), floor_gate(x.y));
    };
    // g, and g_l - g as a sum of its own: gates of -160 add up to -2560, where FP32 has steps of
    // 2^-12
    float2 g = make_float2(0.f, 0.f), tail[kRows];
#pragma unroll 8
    for (int r = 0; r < r0; ++r) g = add2(g, gate(r));
    if (!FROM_START) {
        float2 after = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int r = C - 1; r >= r0 + kRows; --r) after = add2(after, gate(r));
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i) {
            tail[i] = after;
            after = add2(after, gate(r0 + i));
        }
    }
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = r0 + i;
        g = add2(g, gate(r));
        if (FROM_START) tail[i] = make_float2(-g.x, -g.y);
        const float2 q = unpack2<T16>(*reinterpret_cast<const uint32_t *>(&raw.q[r][2 * c2]));
        const float2 k = unpack2<T16>(*reinterpret_cast<const uint32_t *>(&raw.k[r][2 * c2]));
        const float2 up = make_float2(ex2(g.x), ex2(g.y));
        const float2 dn = make_float2(ex2(tail[i].x), ex2(tail[i].y));
        const uint32_t off = plane_off(r, c2 >> 2) + (c2 & 3) * 4;
        const float2 kw = mul2(k, up), kd = mul2(k, dn);
        const float2 qw = mul2(mul2(q, make_float2(scale, scale)), up);
        put_split(planes + KW_HI * kPlane, off, kw.x, kw.y);
        put_split(planes + QW_HI * kPlane, off, qw.x, qw.y);
        put_split(planes + KD_HI * kPlane, off, kd.x, kd.y);
        if (r == C - 1) *reinterpret_cast<float2 *>(&decay[2 * c2]) = up;
        if (FROM_START) big = max_nan(big, max_nan(fabsf(kd.x), fabsf(kd.y)));
    }
    return !(big <= 0x1p96f && g.x >= -100.f && g.y >= -100.f);
}

// hi and lo A-fragments of a 16x16 FP32 block held as two adjacent 16x8 accumulators.
__device__ __forceinline__ void split_frag(const float (&c0)[4], const float (&c1)[4],
                                           uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(c0[0], c0[1], hi[0], lo[0]);
    split2(c0[2], c0[3], hi[1], lo[1]);
    split2(c1[0], c1[1], hi[2], lo[2]);
    split2(c1[2], c1[3], hi[3], lo[3]);
}

// acc[2] (16x16) += A (hi, lo) * B, B's hi and lo fragments of two 8-column tiles.
__device__ __forceinline__ void mma3(float (&c0)[4], float (&c1)[4], const uint32_t (&ah)[4],
                                     const uint32_t (&al)[4], const uint32_t (&bh)[4],
                                     const uint32_t (&bl)[4]) {
    mma16816(c0, ah, bh[0], bh[1]);
    mma16816(c1, ah, bh[2], bh[3]);
    mma16816(c0, ah, bl[0], bl[1]);
    mma16816(c1, ah, bl[2], bl[3]);
    mma16816(c0, al, bh[0], bh[1]);
    mma16816(c1, al, bh[2], bh[3]);
}

// The same for two pairs of tiles with left operands of their own, the four accumulators in
// turn: a product's result is needed again 32 issue cycles later, its latency being 22.
// LO0: the first pair's B has a lo part (inputs that are exact in BF16 have none).
template <bool LO0>
__device__ __forceinline__ void mma3x2(float (&c0)[4], float (&c1)[4], float (&d0)[4],
                                       float (&d1)[4], const uint32_t (&ah)[4],
                                       const uint32_t (&al)[4], const uint32_t (&bh)[4],
                                       const uint32_t (&bl)[4], const uint32_t (&xh)[4],
                                       const uint32_t (&xl)[4], const uint32_t (&yh)[4],
                                       const uint32_t (&yl)[4]) {
    mma16816(c0, ah, bh[0], bh[1]);
    mma16816(c1, ah, bh[2], bh[3]);
    mma16816(d0, xh, yh[0], yh[1]);
    mma16816(d1, xh, yh[2], yh[3]);
    mma16816(c0, al, bh[0], bh[1]);
    mma16816(c1, al, bh[2], bh[3]);
    mma16816(d0, xl, yh[0], yh[1]);
    mma16816(d1, xl, yh[2], yh[3]);
    if (LO0) {
        mma16816(c0, ah, bl[0], bl[1]);
        mma16816(c1, ah, bl[2], bl[3]);
    }
    mma16816(d0, xh, yl[0], yl[1]);
    mma16816(d1, xh, yl[2], yl[3]);
}

// Decay of the accumulators of S^T [16 dv, 128 dk]: columns 16 jj .. 16 jj + 15.
template <int NJ>
__device__ __forceinline__ void decay_cols(float (&S)[NJ][4], const float *decay, int jj, int tc2) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const float2 d = *reinterpret_cast<const float2 *>(&decay[16 * jj + 8 * x + tc2]);
        float(&s)[4] = S[2 * jj + x];
        const float2 u = mul2(make_float2(s[0], s[1]), d);
        const float2 w = mul2(make_float2(s[2], s[3]), d);
        s[0] = u.x; s[1] = u.y; s[2] = w.x; s[3] = w.y;
    }
}

// Per-lane byte offsets of ldmatrix.x4 in a [16][16] tile with 32-byte rows: matrices
// (rows 0-7, cols 0-7), (rows 0-7, cols 8-15), (rows 8-15, cols 0-7), (rows 8-15, cols 8-15).
__device__ __forceinline__ uint32_t tile_lane(int lane) {
    return (uint32_t)(((lane & 7) + ((lane >> 4) & 1) * 8) * 32 + ((lane >> 3) & 1) * 16);
}

// The accumulators of S^T [16 dv, 8 NJ dk] as a checkpoint: 8 dk rows by 16 dv columns a
// block, [dk / 8][dv / 16][32 lanes][16 bytes], a lane's words being (row lane / 4, columns
// 2 (lane % 4), + 1) of the block's left half, hi and lo, and the same of its right half -- the
// accumulator layout of S [dk, dv], whose left-operand fragments sum over dv.
template <int NJ>
__device__ __forceinline__ void store_checkpoint(char *base, const float (&S)[NJ][4], int tile,
                                                 int j0, int lane) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        uint32_t h0, l0, h1, l1;
        split2(S[j][0], S[j][1], h0, l0);
        split2(S[j][2], S[j][3], h1, l1);
        reinterpret_cast<uint4 *>(base)[((j0 + j) * 8 + tile) * 32 + lane] =
            make_uint4(movm_t(h0), movm_t(l0), movm_t(h1), movm_t(l1));
    }
}

__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&w)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}
// A warp's 16 tokens of 16 columns, given transposed (words: tokens 0-7 of columns 0-7 and 8-15,
// tokens 8-15), to rows `row` bytes apart from `at` on, in 16-byte pieces through 512 bytes of
// shared memory: a row's 32 bytes leave together (4-byte stores straight from the transposed
// words cost the walk 200 cycles a step more).  Only `tokens` rows exist; `end` is the size of
// what lies behind `base`.
__device__ __forceinline__ void store_out(char *stage, const uint32_t (&w)[4], char *at, size_t row,
                                          int tokens, const char *base, size_t end, unsigned *dbg,
                                          int lane) {
    auto off = [](int r, int c) { return (uint32_t)(r * 32 + ((c ^ (r >> 2 & 1)) << 4)); };
    stsm4t(tc::smem_u32(stage) + off((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1), w);
    __syncwarp();
    const int r = lane >> 1, c = lane & 1;
    const uint4 u = *reinterpret_cast<const uint4 *>(stage + off(r, c));
    char *to = at + r * row + c * 16;
    if (r < tokens && dbg_ok(dbg, (size_t)(to - base) + 15, end, DBG_STORE))
        *reinterpret_cast<uint4 *>(to) = u;
    __syncwarp();
}

// Moves an accumulator pair's sum away, and adds it again.
__device__ __forceinline__ void take_sum(float (&x)[2][4], float (&kept)[2][4]) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            kept[j][p] = x[j][p];
            x[j][p] = 0.f;
        }
}
__device__ __forceinline__ void add_sum(float (&x)[2][4], const float (&kept)[2][4]) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) x[j][p] += kept[j][p];
}

// The half `second` of an accumulator pair: warps choose without a branch, which would make all
// that follows wait for its lanes to meet again.
__device__ __forceinline__ void half_of(const float (&x)[2][4], bool second, float (&y)[4]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) y[p] = second ? x[1][p] : x[0][p];
}

// A [16 dv, 16 token] accumulator pair as hi/lo planes of rows of tokens, in 8x8 blocks
// [token / 8][dv / 8][8 token][8 dv] of a 64-token slot: eight tokens of it ...
__device__ __forceinline__ void store_row_block(char *base, const float (&x)[4], int block, int dv0,
                                                int lane) {
    uint32_t h0, l0, h1, l1;
    split2(x[0], x[1], h0, l0);
    split2(x[2], x[3], h1, l1);
    char *p = base + ((size_t)block * 16 + dv0 / 8) * 128 + lane * 4;
    *reinterpret_cast<uint32_t *>(p) = movm_t(h0);
    *reinterpret_cast<uint32_t *>(p + 128) = movm_t(h1);
    *reinterpret_cast<uint32_t *>(p + kRowPlane) = movm_t(l0);
    *reinterpret_cast<uint32_t *>(p + kRowPlane + 128) = movm_t(l1);
}
// ... and both eights; t0 is the step's first token in its slot.
__device__ __forceinline__ void store_rows(char *base, const float (&x)[2][4], int t0, int dv0,
                                           int lane) {
    store_row_block(base, x[0], t0 / 8, dv0, lane);
    store_row_block(base, x[1], t0 / 8 + 1, dv0, lane);
}

}  // namespace chunk
}  // namespace kda
