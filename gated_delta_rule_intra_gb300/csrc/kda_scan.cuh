// Shared parts of the selective scan's kernels.  Per channel d a state h of N numbers:
//   D_t = softplus(delta_t + delta_bias),  h_t[n] = exp(D_t A[n]) h_{t-1}[n] + D_t u_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + skip u_t) silu(z_t).
//
// A thread holds four states of each of two channels (N is padded to a power of two, NP; padded ones
// stay zero), NP / 4 neighbouring lanes a channel; half of a CTA's 256 threads walk 1024 / NP channels
// through their tokens in tiles of 16.  What does not depend on the state -- step sizes, inputs,
// the gate -- is prepared and finished by the other half, one tile ahead and one behind, with one
// barrier a tile: each takes eight neighbouring channels of a token.  They
// leave it in shared memory with the tokens last, as they leave B and C: a lane then reads four
// tokens of a number at once, and products of neighbouring tokens are one instruction (f32x2).
// Two channels a thread, because every byte that a lane reads from shared memory costs the same
// whether or not its neighbours read it too: with one channel a thread, B and C alone are 2.5 of the
// 4 cycles that the exponentials leave.  Sums over a channel's states are taken for four tokens at once,
// each lane ending with one token's.
//
// A sequence is one chain; where there are too few channels to fill the card it is cut into
// segments.  A first pass walks them all from zero and leaves each one's end (and the sum of its
// step sizes, which is its decay); the second begins with what the segments in front of it make of
// the first state.
#pragma once

#include "kda_rows.cuh"

namespace kda {
namespace scan {

using namespace rows;

constexpr int kThreads = 128, kTile = kScanTile;
constexpr float kLn2 = 0.6931471805599453f;

template <int NP_> struct Shape {
    static constexpr int NP = NP_, L = NP / 4;           // lanes of a channel
    static constexpr int HC = kThreads / L, CH = 2 * HC;  // a thread has channels c and c + HC of CH
    static constexpr int kChunks = CH / 8;                // of eight channels
    static constexpr int kPer = kTile * kChunks / kThreads > 0 ? kTile * kChunks / kThreads : 1;  // of a thread
    static constexpr int kRow = CH + 8;  // of a [kTile][..] array that lanes write four tokens of
    static constexpr int kBC = (kTile * NP + kThreads - 1) / kThreads;  // elements of B, of C
    static constexpr int kVec = kTile * 4 + 4;  // of an [L][..] array of four states' tokens: parts in other banks
};

// The order of a thread's four states: number i is state n0 + (i ^ turn).  The order changes with the
// channel so that in the sums over a warp's channels that leave each lane with one state's, every
// lane keeps the same of its numbers and sends the same ones.
template <int NP> __device__ __forceinline__ int turn_of(int tid) {
    constexpr int CW = 32 / Shape<NP>::L;  // a warp's channels, side by side
    const int cl = tid % 32 / Shape<NP>::L;
    return CW == 2 ? 0 : CW == 4 ? (cl & 1) << 1 : cl / (CW / 8) & 3;
}

// Where four tokens (4 q ..) of channel c are in a [CH][kTile] array.  The groups of four change
// places with c / 8, so that threads which write one token of channels eight apart meet different
// banks.
__device__ __forceinline__ int place(int c, int q) { return c * kTile + 4 * (q ^ (c >> 3 & 3)); }

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// log(1 + e^x): with t = e^-|x| and s = t / (2 + t), log(1 + t) = 2 artanh(s) as its series, whose
// s^2 is at most 1/9.  Small t keep their accuracy, which log(1 + t) would lose.
__device__ __forceinline__ float2 softplus(float2 x) {
    const float2 t = make_float2(ex2(-kLog2e * fabsf(x.x)), ex2(-kLog2e * fabsf(x.y)));
    const float2 s = mul2(t, make_float2(rcp(2.f + t.x), rcp(2.f + t.y))), q = mul2(s, s);
    float2 r = fma2(q, both(1.f / 13.f), both(1.f / 11.f));
    r = fma2(q, r, both(1.f / 9.f));
    r = fma2(q, r, both(1.f / 7.f));
    r = fma2(q, r, both(1.f / 5.f));
    r = fma2(q, r, both(1.f / 3.f));
    r = fma2(q, r, both(1.f));
    return fma2(add2(s, s), r, make_float2(x.x > 0.f ? x.x : 0.f, x.y > 0.f ? x.y : 0.f));
}
__device__ __forceinline__ float softplus(float x) { return softplus(both(x)).x; }

// v[V] summed over LANES lanes STRIDE apart: every lane ends with V / LANES of the sums (one where
// there are more lanes), the part of them that its place among the lanes says.
template <int LANES, int STRIDE, int V> __device__ __forceinline__ void scatter_sum(float (&v)[V], int lane) {
    if constexpr (LANES > 1) {
        constexpr int off = STRIDE * LANES / 2;
        if constexpr (V > 1) {
            const bool up = lane & off;
            float half[V / 2];
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const float send = up ? v[k] : v[k + V / 2], keep = up ? v[k + V / 2] : v[k];
                half[k] = keep + __shfl_xor_sync(0xffffffffu, send, off);
            }
            scatter_sum<LANES / 2, STRIDE>(half, lane);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) v[k] = half[k];
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
            scatter_sum<LANES / 2, STRIDE>(v, lane);
        }
    }
}

// Which block of channels and which part of which sequence a CTA has.
template <int NP> struct Block {
    int group, c0, channels, slot, blk;  // c0: first channel; slot: the segment; blk: in the group
    Piece p;
    __device__ __forceinline__ Block(const ScanArgs &a, int nb) {
        const unsigned blocks = (unsigned)(nb * a.G), b = blockIdx.x % blocks;
        slot = (int)(blockIdx.x / blocks);
        group = (int)(b / (unsigned)nb);
        blk = (int)(b - (unsigned)group * nb);
        const int per = a.D / a.G, at = blk * Shape<NP>::CH;
        c0 = group * per + at;
        channels = min(Shape<NP>::CH, per - at);
        p = find_piece(a.tok, slot, a.segment);
    }
    // The first of the sequence's slots in `saved`.
    __device__ __forceinline__ long long tiles0(const ScanArgs &a) const {
        return a.tok.cu_seqlens ? p.row0 / kTile + p.seq
                                : (long long)p.seq * (a.tok.T > kTile ? (a.tok.T + kTile - 1) / kTile : 1);
    }
};

template <typename T>
__device__ __forceinline__ void store_chunk(void *base, long long stride, long long row, int c,
                                            int left, const Vec<T, 8> &x, int unit) {
    T *at = (T *)base + row * stride + c;
    constexpr int E = sizeof(T);
    if (unit == 16) {
#pragma unroll
        for (int i = 0; i < 8; i += 16 / E)
            if (i < left) *(uint4 *)(at + i) = *(const uint4 *)(x.v + i);
    } else if (unit == 8) {
#pragma unroll
        for (int i = 0; i < 8; i += 8 / E)
            if (i < left) *(uint2 *)(at + i) = *(const uint2 *)(x.v + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) at[i] = x.v[i];
    }
}
// The row of what the gate multiplies, FP32, rows on 16-byte boundaries.
__device__ __forceinline__ float *open_row(const ScanArgs &a, long long row) {
    return a.open + row * (long long)((a.D + 3) / 4 * 4);
}
template <typename T> __device__ __forceinline__ float2 pair(const Vec<T, 8> &x, int i) { return x.two(2 * i); }
template <typename T> __device__ __forceinline__ void put_pair(Vec<T, 8> &x, int i, float2 v) {
    x.put(2 * i, v);
}
__device__ __forceinline__ float2 sigmoid2(float2 x) { return make_float2(sigmoid(x.x), sigmoid(x.y)); }

// A tile's elements of B or C in the registers of all threads, and from there to shared memory.
template <typename T, int NP> struct Vectors {
    using S = Shape<NP>;
    T v[S::kBC];
    __device__ __forceinline__ void load(int tid, const void *base, long long stride, long long row0,
                                         int rows, int group, int N) {
#pragma unroll
        for (int i = 0; i < S::kBC; ++i) {
            const int e = tid + i * kThreads, t = e / NP, n = e % NP;
            v[i] = t < rows && n < N ? ((const T *)base)[(row0 + t) * stride + (long long)group * N + n]
                                     : from_f32<T>(0.f);
        }
    }
    __device__ __forceinline__ void put(int tid, float (*to)[S::kVec]) const {  // [L][state][token]
#pragma unroll
        for (int i = 0; i < S::kBC; ++i) {
            const int e = tid + i * kThreads;
            if (S::kBC * kThreads == kTile * NP || e < kTile * NP) to[e % NP / 4][e % 4 * kTile + e / NP] = as_f32(v[i]);
        }
    }
};

// A thread's four numbers of a [.., D, N] tensor of states (or of A).
struct Four {
    float2 lo, hi;
    __device__ __forceinline__ float get(int i) const { return i == 0 ? lo.x : i == 1 ? lo.y : i == 2 ? hi.x : hi.y; }
};
__device__ __forceinline__ Four four(float4 x) { return {make_float2(x.x, x.y), make_float2(x.z, x.w)}; }
__device__ __forceinline__ float4 one(Four x) { return make_float4(x.lo.x, x.lo.y, x.hi.x, x.hi.y); }
// (`turn`: number i is state n + (i ^ turn))
__device__ __forceinline__ Four load_states(const float *base, size_t channel, int n, int N, bool ok, int turn = 0) {
    float v[4] = {};
    if (ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + (i ^ turn) < N) v[i] = base[channel * N + n + (i ^ turn)];
    }
    return {make_float2(v[0], v[1]), make_float2(v[2], v[3])};
}
__device__ __forceinline__ void store_states(float *base, size_t channel, int n, int N, Four x, int turn = 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + (i ^ turn) < N) base[channel * N + n + (i ^ turn)] = x.get(i);
}
using kda::fma2;
using kda::mul2;

// A number twice, as one operand of paired operations that stays where it is (the compiler would
// copy it together anew for each: an instruction of eight).
__device__ __forceinline__ uint64_t twice(float x) {
    uint64_t r;
    asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, uint64_t b) {
    float2 r;
    asm("{\n.reg .b64 x;\nmov.b64 x, {%2, %3};\nmul.rn.f32x2 x, x, %4;\nmov.b64 {%0, %1}, x;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "l"(b));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, uint64_t b, float2 c) {
    float2 r;
    asm("{\n.reg .b64 x, z;\nmov.b64 x, {%2, %3};\nmov.b64 z, {%5, %6};\nfma.rn.f32x2 x, x, %4, z;\n"
        "mov.b64 {%0, %1}, x;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "l"(b), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ Four scaled(Four a, float x) { return {mul2(a.lo, both(x)), mul2(a.hi, both(x))}; }
__device__ __forceinline__ float2 fma2(float2 a, uint64_t b, uint64_t c) {
    float2 r;
    asm("{\n.reg .b64 x;\nmov.b64 x, {%2, %3};\nfma.rn.f32x2 x, x, %4, %5;\nmov.b64 {%0, %1}, x;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "l"(b), "l"(c));
    return r;
}
// The argument of a token's decay, d A log2(e), is taken a little larger than that: the exponential unit's
// results are too small on the mean, and a state adds that up over all tokens that it lasts.  Measured, for
// arguments of a size in [1, 2) times 2^n, in 1e-8: n = -20 .. -15 0.7 to 1.1, -14 .. -9 0.5 to 0.9, -8 1.5 and
// 2.2, -7 3.1 and 2.2, -6 2.2 and 2.9, -5 2.7 and 0.7, -4 .. -1 1.4 to 2.8.  So 2.5e-8 (1.7e-8 of the result), or
// 1e-8 where the slowest of a thread's states is below 2^-8, of which no more than 0.3e-8 a token
// is left.  2^0 is still 1.  Relative error of the final states of 8192 tokens, A from -0.001 to -1: 3.5e-6;
// 3.9e-5 with 2.5e-8 for all, 2.6e-5 without.  (What is left of a step size that never changes is the unit's
// rounding of that one decay, up to 8e-8 a token.)
constexpr float kQuick = 2.5e-8f, kSlow = 1e-8f;
// e: the smallest size of a thread's arguments.
__device__ __forceinline__ float raise_of(float e) { return e < 0x1p-8f ? kSlow : kQuick; }
__device__ __forceinline__ float slowest_of(Four A2, int n, int N, int turn) {
    float x = 3e38f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + (i ^ turn) < N) x = fminf(x, fabsf(A2.get(i)));
    return x;
}
// That number for each of the forward's walking threads, from the first token of the tile that was walked before:
// the preparing half finds it, because the walking threads have no register left for it (found there, a prompt
// of 32768 tokens takes 1290 us instead of 1249).
template <int NP> struct Raise {
    float slowest[2];
    int at[2];
    __device__ __forceinline__ Raise(const ScanArgs &a, int c0, int channels, int tid) {
        using S = Shape<NP>;
        const int n0 = 4 * (tid % S::L);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = tid / S::L + j * S::HC;
            slowest[j] = slowest_of(scaled(load_states(a.A, (size_t)c0 + c, n0, a.N, c < channels), kLog2e), n0,
                                    c < channels ? a.N : 0, 0);
            at[j] = place(c, 0);
        }
    }
    __device__ __forceinline__ float2 next(const float *d) const {
        return both(raise_of(fminf(fabsf(d[at[0]]) * slowest[0], fabsf(d[at[1]]) * slowest[1])));
    }
};
// The first pass over segments keeps to 2.5e-8: its sums are a segment's alone.
__device__ __forceinline__ float2 exponent(float2 d, uint64_t A) { return fma2(d, A, both(kQuick)); }
// 2^(d a)
__device__ __forceinline__ Four decay(float2 dd, Four a2, float raise) {
    const float2 l = fma2(dd, a2.lo, both(raise)), h = fma2(dd, a2.hi, both(raise));
    return {make_float2(ex2(l.x), ex2(l.y)), make_float2(ex2(h.x), ex2(h.y))};
}
__device__ __forceinline__ Four mul(Four a, Four b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ Four fma(Four a, Four b, Four c) { return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)}; }
__device__ __forceinline__ Four fma(float2 a, Four b, Four c) { return {fma2(a, b.lo, c.lo), fma2(a, b.hi, c.hi)}; }
__device__ __forceinline__ Four mul(float2 a, Four b) { return {mul2(a, b.lo), mul2(a, b.hi)}; }
__device__ __forceinline__ float dot(Four a, Four b) {
    const float2 s = fma2(a.hi, b.hi, mul2(a.lo, b.lo));
    return s.x + s.y;
}

// Shared memory that the phase behind a barrier only reads: the loads are plain functions of their
// address, so that no store of the phase holds them back (it is not known that the arrays are
// apart); `phase`, which is new behind every barrier, keeps them from moving across it.
struct Phase {
    uint32_t base;
    __device__ __forceinline__ Phase(const void *smem) : base((uint32_t)__cvta_generic_to_shared(smem)) {}
    __device__ __forceinline__ void next() { asm volatile("" : "+r"(base)::"memory"); }
    __device__ __forceinline__ void load4(uint32_t off, float2 (&to)[2]) const {
        asm("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
            : "=f"(to[0].x), "=f"(to[0].y), "=f"(to[1].x), "=f"(to[1].y) : "r"(base + off));
    }
    __device__ __forceinline__ float load(uint32_t off) const {
        float x;
        asm("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(base + off));
        return x;
    }
    __device__ __forceinline__ uint64_t load_pair(uint32_t off) const {
        uint64_t x;
        asm("ld.shared.b64 %0, [%1];" : "=l"(x) : "r"(base + off));
        return x;
    }
    __device__ __forceinline__ float2 load2(uint32_t off) const {
        float2 x;
        asm("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(base + off));
        return x;
    }
};
// All 2 kThreads of a CTA, and the kThreads of its second half.
__device__ __forceinline__ void sync_all() { asm volatile("bar.sync 0, %0;" ::"n"(2 * kThreads) : "memory"); }
__device__ __forceinline__ void sync_half() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// How the four sums that scatter_sum<L, 1> leaves are spread: a lane's first token, and how many.
template <int L> struct Share {
    static constexpr int kCount = L < 4 ? 4 / L : 1;
    static __device__ __forceinline__ int first(int part) { return L < 4 ? part * kCount : part / (L / 4 > 0 ? L / 4 : 1); }
    static __device__ __forceinline__ bool mine(int part) { return L <= 4 || part % (L / 4 > 0 ? L / 4 : 1) == 0; }
};

struct Unit : rows::Boundary {
    Unit(const ScanArgs &a) : rows::Boundary(esize(a.dtype), a.D / a.G) {}
};

}  // namespace scan
}  // namespace kda
