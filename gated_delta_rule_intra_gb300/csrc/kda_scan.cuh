// Shared parts of the selective scan's kernels.  Per channel d a state h of N numbers:
//   D_t = softplus(delta_t + delta_bias),  h_t[n] = exp(D_t A[n]) h_{t-1}[n] + D_t u_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + skip u_t) silu(z_t).
//
// A thread holds four states of a channel (N is padded to a power of two, NP; padded ones stay
// zero), NP / 4 neighbouring lanes a channel.  A CTA of 128 threads walks 512 / NP channels through
// its tokens in tiles of 16: the tile's step sizes and inputs are prepared by threads that each
// take four neighbouring channels of one token (8-byte loads), and come to the lanes that need them
// through shared memory, as do B and C; sums over a channel's states are taken for four
// tokens at once, each lane ending with one token's.
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
    static constexpr int NP = NP_, L = NP / 4, CH = kThreads / L;  // lanes of a channel, channels
    static constexpr int kQuads = CH / 4;                          // of four channels
    static constexpr int kPer = (kTile * kQuads + kThreads - 1) / kThreads;  // quads of a thread
    static constexpr int kRow = CH + 8;  // of a [kTile][..] array that lanes write four tokens of
    static constexpr int kBC = (kTile * NP + kThreads - 1) / kThreads;  // elements of B, of C
};

// log(1 + e^x): with t = e^-|x| and s = t / (2 + t), log(1 + t) = 2 artanh(s) as its series, whose
// s^2 is at most 1/9.  Small t keep their accuracy, which log(1 + t) would lose.
__device__ __forceinline__ float softplus(float x) {
    const float t = ex2(-kLog2e * fabsf(x)), s = t * rcp(2.f + t), q = s * s;
    float r = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    r = fmaf(q, r, 1.f / 9.f);
    r = fmaf(q, r, 1.f / 7.f);
    r = fmaf(q, r, 1.f / 5.f);
    r = fmaf(q, r, 1.f / 3.f);
    r = fmaf(q, r, 1.f);
    return fmaf(2.f * s, r, x > 0.f ? x : 0.f);
}

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

// Four neighbouring channels of a token; zeros where there are none.  `vec`: rows begin on
// boundaries of four elements and blocks hold whole quads.
template <typename T>
__device__ __forceinline__ Vec<T, 4> load_quad(const void *base, long long stride, long long row,
                                               int c, int left, bool ok, bool vec) {
    Vec<T, 4> x;
    x.clear();
    const T *at = (const T *)base + row * stride + c;
    if (vec) {
        if (ok && left > 0) x = *reinterpret_cast<const Vec<T, 4> *>(at);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (ok && i < left) x.v[i] = at[i];
    }
    return x;
}
template <typename T>
__device__ __forceinline__ void store_quad(void *base, long long stride, long long row, int c,
                                           int left, const Vec<T, 4> &x, bool vec) {
    T *at = (T *)base + row * stride + c;
    if (vec) {
        if (left > 0) *reinterpret_cast<Vec<T, 4> *>(at) = x;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) at[i] = x.v[i];
    }
}

// A tile's elements of B or C in the registers of all threads, and from there to shared memory.
template <typename T, int NP> struct Vectors {
    using S = Shape<NP>;
    T v[S::kBC];
    __device__ __forceinline__ void load(const void *base, long long stride, long long row0, int rows,
                                         int group, int N) {
#pragma unroll
        for (int i = 0; i < S::kBC; ++i) {
            const int e = threadIdx.x + i * kThreads, t = e / NP, n = e % NP;
            v[i] = t < rows && n < N ? ((const T *)base)[(row0 + t) * stride + (long long)group * N + n]
                                     : from_f32<T>(0.f);
        }
    }
    __device__ __forceinline__ void put(float (*to)[NP]) const {
#pragma unroll
        for (int i = 0; i < S::kBC; ++i) {
            const int e = threadIdx.x + i * kThreads;
            if (S::kBC * kThreads == kTile * NP || e < kTile * NP) to[e / NP][e % NP] = as_f32(v[i]);
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
__device__ __forceinline__ Four load_states(const float *base, size_t channel, int n, int N, bool ok) {
    float v[4] = {};
    if (ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) v[i] = base[channel * N + n + i];
    }
    return {make_float2(v[0], v[1]), make_float2(v[2], v[3])};
}
__device__ __forceinline__ void store_states(float *base, size_t channel, int n, int N, Four x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < N) base[channel * N + n + i] = x.get(i);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ Four scaled(Four a, float x) { return {mul2(a.lo, both(x)), mul2(a.hi, both(x))}; }
// 2^(d a)
__device__ __forceinline__ Four decay(float2 dd, Four a2) {
    const float2 l = mul2(dd, a2.lo), h = mul2(dd, a2.hi);
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

// How the four sums that scatter_sum<L, 1> leaves are spread: a lane's first token, and how many.
template <int L> struct Share {
    static constexpr int kCount = L < 4 ? 4 / L : 1;
    static __device__ __forceinline__ int first(int part) { return L < 4 ? part * kCount : part / (L / 4 > 0 ? L / 4 : 1); }
    static __device__ __forceinline__ bool mine(int part) { return L <= 4 || part % (L / 4 > 0 ? L / 4 : 1) == 0; }
};

inline bool vec_ok(const ScanArgs &a, const void *p, long long stride) {
    return !p || (aligned(p, 4 * (size_t)esize(a.dtype)) && stride % 4 == 0);
}

}  // namespace scan
}  // namespace kda
