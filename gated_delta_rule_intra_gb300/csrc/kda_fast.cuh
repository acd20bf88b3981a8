// The recurrence kernels for BF16 training (no state taken or returned): the same walk as in
// kda_chunk.cuh with one FP16 product where the others take three BF16 ones.
//
// o and the gradients leave as BF16 (8 bits), so operands of 11 bits are enough: a rounding of
// 2^-12 a product hides behind the outputs' 2^-9.  FP16 has the bits but not FP32's range, so
// operands that a user may scale freely carry a power of two of their own: the state tile of a
// warp is held in FP32 as S c with |S c| <= 2^15 (c follows from a running bound, made exact
// again whenever it runs out), e and the gradients a power of two per tile and step found
// with a warp reduction, and the planes of q and k one each that follows a step's largest |q| and
// |k|: an input keeps its 11 bits down to 2^-6 of that where the gates are mild, 2^-11 otherwise.
// Steps whose inputs pass 2^14, or anything not finite, take the definition token by token in FP32
// instead.  Sums, the state, the solve and the pairs' scores stay FP32 (the small [16][16]
// products and the scores take TF32 operands, which need no range).
#pragma once

#include "kda_chunk.cuh"

namespace kda {
namespace fast {

using chunk::C;
using chunk::D;
using chunk::kPlane;

constexpr int kHalf = 128;        // threads of each half of the preparing warps
constexpr int kTall = C * C * 4;  // bytes of an FP32 [16][16] tile
constexpr int kTile = C * C * 2;
// Per slot of 64 tokens and head: the state at its start, e or Y, T^T and P^T of its steps, and
// the scales of the first two: [8 tiles] and [4 steps][8 tiles].
constexpr size_t kCkptBytes = D * D * 2, kRowsBytes = BT * D * 2, kTilesBytes = 4 * 2 * kTall;
constexpr int kScales = 40;
constexpr float kLimit = 32768.f;  // |S c| while it is an operand
constexpr int kFresh = 2;          // exponent of the largest |S c| after a renewal: far below
                                   // the limit, so that the bound lasts for some 100 steps
constexpr int kTop = 13;           // exponent of other operands' largest element

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
// A 16x8 accumulator as left operand of a TF32 product: the fragment's elements t and t + 4 of
// the summed dimension are the accumulator's neighbouring columns 2t and 2t + 1, so the right
// operands hold the even elements of each eight before the odd ones (tall_at()).
__device__ __forceinline__ void tf_frag(const float (&c)[4], uint32_t (&a)[4]) {
    a[0] = to_tf32(c[0]);
    a[1] = to_tf32(c[2]);
    a[2] = to_tf32(c[1]);
    a[3] = to_tf32(c[3]);
}
// FP32 [16][16] tile: 64-byte rows of four 16-byte chunks (elements 0 2 4 6, 1 3 5 7, 8 10 12
// 14, 9 11 13 15), swizzled by the row.
__device__ __forceinline__ uint32_t tall_off(int r, int chunk) {
    return (uint32_t)(r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4));
}
__device__ __forceinline__ uint32_t tall_at(int r, int c) {
    return tall_off(r, (c >> 3) * 2 + (c & 1)) + ((c & 7) >> 1) * 4;
}
// Right operands of a whole tile: rows 0-7 and 8-15 as columns, the rows' elements summed.
__device__ __forceinline__ void load_tall(uint32_t tile, int lane, uint32_t (&lo)[4],
                                          uint32_t (&hi)[4]) {
    const uint32_t a = tile + tall_off(lane & 7, lane >> 3);
    chunk::ldsm4(lo, a);
    chunk::ldsm4(hi, a + 8 * 64);
}
// acc (two 8-column tiles) += X B, X given as its two 16x8 accumulators.
__device__ __forceinline__ void mma_tall(float (&c0)[4], float (&c1)[4], const uint32_t (&x0)[4],
                                         const uint32_t (&x1)[4], const uint32_t (&lo)[4],
                                         const uint32_t (&hi)[4]) {
    mma_tf32(c0, x0, lo[0], lo[1]);
    mma_tf32(c1, x0, hi[0], hi[1]);
    mma_tf32(c0, x1, lo[2], lo[3]);
    mma_tf32(c1, x1, hi[2], hi[3]);
}

using chunk::max_nan;
// The warp's largest of non-negative values (or of their bits); NaN counts as largest.
__device__ __forceinline__ float warp_max(float x) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}
__device__ __forceinline__ float abs_max(const float (&x)[2][4]) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) m = max_nan(m, fabsf(x[j][p]));
    return m;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// The power of two that brings `largest` to an exponent of `target`, and its inverse.
__device__ __forceinline__ float scale_for(float largest, int target) {
    const int e = max((int)(__float_as_uint(largest) >> 23 & 0xff), target + 1);
    return __uint_as_float((uint32_t)(254 + target - min(e, 254)) << 23);
}
__device__ __forceinline__ float inverse_of(float power) {
    return __uint_as_float((254u << 23) - __float_as_uint(power));
}

// A warp's state tile: S^T [16 dv, 128 dk] times c.
struct Tile {
    float s[16][4];
    float c, inv, bound;  // |s| <= bound

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < 16; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        c = inv = 1.f;
        bound = 0.f;
    }
    // The scale that goes with the tile when it is saved: none to respect where it is zero.
    __device__ __forceinline__ float saved_scale() const { return bound == 0.f ? 0x1p100f : c; }
    // The exact largest element back to 2^2 (ignoring what is not finite).
    __device__ __forceinline__ void renew() {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float x = fabsf(s[j][p]);
                m = fmaxf(m, x <= 3.4e38f ? x : 0.f);
            }
        m = warp_max(m);
        // c itself within 2^-100 .. 2^100: a state outside these has left FP16's reach
        float f = m > 0.f ? scale_for(m, kFresh) : 1.f;
        if (c * f > 0x1p100f || c * f < 0x1p-100f) f = 1.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p) s[j][p] *= f;
        c *= f;
        inv = inverse_of(c);
        bound = m * f;
    }
};

// Where a step's raw inputs lie in shared memory; q and k rows are padded, so that eight rows
// at the same channel fall into different banks.
constexpr int kRowPad = D + 8;
struct __align__(16) RawStage {
    uint16_t q[C][kRowPad];
    uint16_t k[C][kRowPad];
    float gate[C][D];
};

__device__ __forceinline__ float2 bf2(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ float bf1(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// FP16 planes of a step, rows of tokens (chunk::plane_off).
struct __align__(128) Planes {
    char kw[kPlane], qw[kPlane], kd[kPlane];
    float decay[D];     // 2^g_l
    uint32_t kmax[4];   // |k|, |q| of each preparing warp's rows: BF16 bits shifted up
    uint32_t qmax[4];
    float kinv, qinv;   // the planes' powers of two, inverse
    float ktop, qtop;   // backward: the step's largest |k| and |scale q|
    float bmax;         // largest |beta|
    int careful;        // take the definition
};
__device__ __forceinline__ float largest(const uint32_t (&m)[4]) {
    return __uint_as_float(max(max(m[0], m[1]), max(m[2], m[3])));
}

// The power of two that brings a step's largest |k| (or |scale q|) to 1 .. 2, so that the planes
// have FP16's bits for inputs of any size; 1 where there are only zeros.  Outside 2^-60 .. 2^14 it
// stays what it is at the end: what is smaller has no bits beside a value of ordinary size, and
// larger inputs take the definition.
__device__ __forceinline__ float plane_scale(float largest) {
    return largest == 0.f ? 1.f : scale_for(fminf(fmaxf(largest, 0x1p-60f), 0x1p14f), 0);
}
// Where the largest |k| and |scale q| have to be with the planes' powers of two, so that the
// forward may go on with the step before's: finding the maximum in front of the planes would cost
// its preparing warps, whose chain is the longer one, 3% of a mild step and 10% of another.
constexpr float kLeast = 0.125f, kMost = 3.5f;

// The planes' powers of two: kw and kd are taken `k` times as large, qw `q` times.
struct Scales {
    float k = 1.f, q = 1.f;

    __device__ __forceinline__ void follow(const Planes &p, float scale) {
        k = plane_scale(largest(p.kmax));
        q = plane_scale(fabsf(scale) * largest(p.qmax));
    }
    // Zeros fit any power (unused channels, tokens behind the end).
    __device__ __forceinline__ bool in_range(float kmax, float qmax, float scale) const {
        const float x = k * kmax, y = fabsf(scale * q) * qmax;
        return (x >= kLeast || x == 0.f) && x <= kMost && (y >= kLeast || y == 0.f) && y <= kMost;
    }
    __device__ __forceinline__ bool fit(const Planes &p, float scale) const {
        return in_range(largest(p.kmax), largest(p.qmax), scale);
    }
    __device__ __forceinline__ void put(Planes &p) const {
        p.kinv = inverse_of(k);
        p.qinv = inverse_of(q);
    }
};
// A preparing warp's largest |k| and |q| from its threads'; returns whether they are in range.
__device__ __forceinline__ bool put_largest(Planes &out, uint32_t km, uint32_t qm, const Scales &sc,
                                            float scale, int tid) {
    const uint32_t kb = __reduce_max_sync(0xffffffffu, max(km << 16, km & 0xffff0000u));
    const uint32_t qb = __reduce_max_sync(0xffffffffu, max(qm << 16, qm & 0xffff0000u));
    if ((tid & 31) == 0) {
        out.kmax[tid >> 5] = kb;
        out.qmax[tid >> 5] = qb;
    }
    return sc.in_range(__uint_as_float(kb), __uint_as_float(qb), scale);
}

// The largest |q| and |k| among what a preparing thread has copied itself (eight channels of the
// rows tid / 16 and 8 more), which it may read before the others' copies are visible to it: the
// maxima then cost no barrier of their own.
__device__ __forceinline__ void find_largest(const RawStage &raw, Planes &out, int tid) {
    auto most = [&](const uint16_t (*rows)[kRowPad]) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 x =
                *reinterpret_cast<const uint4 *>(&rows[(tid >> 4) + 8 * i][(tid & 15) * 8]);
            m = __vmaxu2(__vmaxu2(m, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
            m = __vmaxu2(__vmaxu2(m, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
        }
        return __reduce_max_sync(0xffffffffu, max(m << 16, m & 0xffff0000u));
    };
    const uint32_t q = most(raw.q), k = most(raw.k);
    if ((tid & 31) == 0) {
        out.qmax[tid >> 5] = q;
        out.kmax[tid >> 5] = k;
    }
}

// Inputs that FP16 planes take; the others go the definition's way.
__device__ __forceinline__ bool in_reach(const Planes &p, float scale) {
    return largest(p.kmax) <= 16384.f && fabsf(scale) * largest(p.qmax) <= 16384.f;
}

// Steps whose channels lose no more than 2^-19 (the mild ones): q 2^g, k 2^g and k 2^-g of inputs
// with a largest element of 1 .. 2 all fit FP16's normal range when the first two are taken 2^14
// times and the last 2^-5 times as large.  The scores are then products of these planes, and the
// key plane is that from the step's start, as in the precise kernels.
constexpr float kMildGate = -19.f;
constexpr int kUp = 14, kMildDown = 5;

// These planes (128 threads, two channels of eight rows each).  Returns whether the step is mild,
// with inputs in range of the planes' powers of two, as far as the thread and its warp have seen.
__device__ __forceinline__ bool prepare_mild(const RawStage &raw, Planes &out, const Scales &sc,
                                             float scale, int tid) {
    const int c2 = tid & 63, r0 = (tid >> 6) * 8;
    auto gate = [&](int r) {
        const float2 x = *reinterpret_cast<const float2 *>(&raw.gate[r][2 * c2]);
        return make_float2(chunk::floor_gate(x.x), chunk::floor_gate(x.y));
    };
    float2 g = make_float2(0.f, 0.f);
    if (r0) {
#pragma unroll
        for (int r = 0; r < 8; ++r) g = chunk::add2(g, gate(r));
    }
    const float2 ks = make_float2(sc.k, sc.k);
    const float2 qs = make_float2(scale * sc.q, scale * sc.q);
    uint32_t km = 0, qm = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + i;
        g = chunk::add2(g, gate(r));
        const uint32_t qr = *reinterpret_cast<const uint32_t *>(&raw.q[r][2 * c2]);
        const uint32_t kr = *reinterpret_cast<const uint32_t *>(&raw.k[r][2 * c2]);
        km = __vmaxu2(km, kr & 0x7fff7fffu);
        qm = __vmaxu2(qm, qr & 0x7fff7fffu);
        const float2 k = chunk::mul2(bf2(kr), ks), q = chunk::mul2(bf2(qr), qs);
        const float2 up = make_float2(ex2(g.x + kUp), ex2(g.y + kUp));
        const float2 dn = make_float2(ex2(-kMildDown - g.x), ex2(-kMildDown - g.y));
        const float2 kw = chunk::mul2(k, up), qw = chunk::mul2(q, up), kd = chunk::mul2(k, dn);
        const uint32_t off = chunk::plane_off(r, c2 >> 2) + (c2 & 3) * 4;
        *reinterpret_cast<uint32_t *>(out.kw + off) = pack_f16(kw.x, kw.y);
        *reinterpret_cast<uint32_t *>(out.qw + off) = pack_f16(qw.x, qw.y);
        *reinterpret_cast<uint32_t *>(out.kd + off) = pack_f16(kd.x, kd.y);
    }
    if (r0) *reinterpret_cast<float2 *>(&out.decay[2 * c2]) = make_float2(ex2(g.x), ex2(g.y));
    return put_largest(out, km, qm, sc, scale, tid) && g.x >= kMildGate && g.y >= kMildGate;
}

// What a thread of prepare() has seen: a channel loses more than 2^-96; none more than a mild step's;
// its warp's inputs are in range of the planes' powers of two.
struct Seen {
    bool strong, mild, in_range;
};
// The operand planes in general (128 threads), kw and qw 2^UP and kd 2^DOWN times as large.
// FORWARD: the cumulative gate too (plus UP, which its differences do not see), and the largest
// inputs, which have been found before otherwise.
template <bool FORWARD, int UP, int DOWN>
__device__ __forceinline__ Seen prepare(const RawStage &raw, Planes &out, float (*gcum)[kRowPad],
                                        const Scales &sc, float scale, int tid) {
    const int c2 = tid & 63, r0 = (tid >> 6) * 8;
    auto gate = [&](int r) {
        const float2 x = *reinterpret_cast<const float2 *>(&raw.gate[r][2 * c2]);
        return make_float2(chunk::floor_gate(x.x), chunk::floor_gate(x.y));
    };
    float2 g = make_float2(0.f, 0.f), total = g;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        if (r == r0) g = total;
        total = chunk::add2(total, gate(r));
    }
    g = chunk::add2(g, make_float2(UP, UP));
    const float2 last = chunk::add2(total, make_float2(UP + DOWN, UP + DOWN));
    const float2 ks = make_float2(sc.k, sc.k);
    const float2 qs = make_float2(scale * sc.q, scale * sc.q);
    uint32_t km = 0, qm = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + i;
        g = chunk::add2(g, gate(r));
        if (FORWARD) *reinterpret_cast<float2 *>(&gcum[r][2 * c2]) = g;
        const uint32_t qr = *reinterpret_cast<const uint32_t *>(&raw.q[r][2 * c2]);
        const uint32_t kr = *reinterpret_cast<const uint32_t *>(&raw.k[r][2 * c2]);
        if (FORWARD) {
            km = __vmaxu2(km, kr & 0x7fff7fffu);
            qm = __vmaxu2(qm, qr & 0x7fff7fffu);
        }
        const float2 q = chunk::mul2(bf2(qr), qs), k = chunk::mul2(bf2(kr), ks);
        const float2 up = make_float2(ex2(g.x), ex2(g.y));
        const float2 dn = make_float2(ex2(last.x - g.x), ex2(last.y - g.y));
        const float2 kw = chunk::mul2(k, up), qw = chunk::mul2(q, up), kd = chunk::mul2(k, dn);
        const uint32_t off = chunk::plane_off(r, c2 >> 2) + (c2 & 3) * 4;
        *reinterpret_cast<uint32_t *>(out.kw + off) = pack_f16(kw.x, kw.y);
        *reinterpret_cast<uint32_t *>(out.qw + off) = pack_f16(qw.x, qw.y);
        *reinterpret_cast<uint32_t *>(out.kd + off) = pack_f16(kd.x, kd.y);
    }
    if (r0 == 8)
        *reinterpret_cast<float2 *>(&out.decay[2 * c2]) = make_float2(ex2(total.x), ex2(total.y));
    return {total.x < -96.f || total.y < -96.f, total.x >= kMildGate && total.y >= kMildGate,
            !FORWARD || put_largest(out, km, qm, sc, scale, tid)};
}

// A step token by token from the definition, forwards: e and o (before its rounding) of a tile
// in accumulator layout, the tile's state updated.
__device__ __forceinline__ void walk_tokens(Tile &t, float (&o)[2][4], float (&e)[2][4],
                                            const RawStage &raw, const float *beta,
                                            const uint16_t (*v)[D], int vcol, float scale,
                                            int lane) {
    const int gr = lane >> 2, tc2 = (lane & 3) * 2;
#pragma unroll 1
    for (int r = 0; r < C; ++r) {
        float u0 = 0.f, u1 = 0.f, w0 = 0.f, w1 = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int ch = 8 * j + tc2;
            const float2 g = *reinterpret_cast<const float2 *>(&raw.gate[r][ch]);
            const float2 k = bf2(*reinterpret_cast<const uint32_t *>(&raw.k[r][ch]));
            const float ax = ex2(chunk::floor_gate(g.x)), ay = ex2(chunk::floor_gate(g.y));
            t.s[j][0] *= ax; t.s[j][1] *= ay; t.s[j][2] *= ax; t.s[j][3] *= ay;
            u0 += k.x * t.s[j][0] + k.y * t.s[j][1];
            u1 += k.x * t.s[j][2] + k.y * t.s[j][3];
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            u0 += __shfl_xor_sync(0xffffffffu, u0, off);
            u1 += __shfl_xor_sync(0xffffffffu, u1, off);
        }
        auto value = [&](int d) {
            const int c = vcol + d;
            return bf1(*reinterpret_cast<const uint16_t *>(
                (const char *)v + chunk::plane_off(r, c >> 3) + (c & 7) * 2));
        };
        const float e0 = value(gr) - u0 * t.inv, e1 = value(gr + 8) - u1 * t.inv;
        const float n0 = beta[r] * e0 * t.c, n1 = beta[r] * e1 * t.c;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int ch = 8 * j + tc2;
            const float2 k = bf2(*reinterpret_cast<const uint32_t *>(&raw.k[r][ch]));
            const float2 q = bf2(*reinterpret_cast<const uint32_t *>(&raw.q[r][ch]));
            t.s[j][0] += k.x * n0; t.s[j][1] += k.y * n0;
            t.s[j][2] += k.x * n1; t.s[j][3] += k.y * n1;
            w0 += q.x * t.s[j][0] + q.y * t.s[j][1];
            w1 += q.x * t.s[j][2] + q.y * t.s[j][3];
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            w0 += __shfl_xor_sync(0xffffffffu, w0, off);
            w1 += __shfl_xor_sync(0xffffffffu, w1, off);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (8 * j + tc2 + (p & 1) == r) {
                    e[j][p] = p < 2 ? e0 : e1;
                    o[j][p] = scale * t.inv * (p < 2 ? w0 : w1);
                }
    }
    t.bound = 2.f * kLimit;  // found again before the next step
}

// The same backwards, for the state's gradient: Y of a tile; dov are the tile's rows of do.
__device__ __forceinline__ void walk_tokens_back(Tile &t, float (&y)[2][4], const RawStage &raw,
                                                 const float *beta, const uint16_t (*dov)[D],
                                                 int vcol, float scale, int lane) {
    const int gr = lane >> 2, tc2 = (lane & 3) * 2;
#pragma unroll 1
    for (int r = C - 1; r >= 0; --r) {
        auto value = [&](int d) {
            const int c = vcol + d;
            return bf1(*reinterpret_cast<const uint16_t *>(
                (const char *)dov + chunk::plane_off(r, c >> 3) + (c & 7) * 2));
        };
        const float o0 = scale * t.c * value(gr), o1 = scale * t.c * value(gr + 8);
        float u0 = 0.f, u1 = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int ch = 8 * j + tc2;
            const float2 k = bf2(*reinterpret_cast<const uint32_t *>(&raw.k[r][ch]));
            const float2 q = bf2(*reinterpret_cast<const uint32_t *>(&raw.q[r][ch]));
            t.s[j][0] += q.x * o0; t.s[j][1] += q.y * o0;
            t.s[j][2] += q.x * o1; t.s[j][3] += q.y * o1;
            u0 += k.x * t.s[j][0] + k.y * t.s[j][1];
            u1 += k.x * t.s[j][2] + k.y * t.s[j][3];
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            u0 += __shfl_xor_sync(0xffffffffu, u0, off);
            u1 += __shfl_xor_sync(0xffffffffu, u1, off);
        }
        const float n0 = beta[r] * u0, n1 = beta[r] * u1;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int ch = 8 * j + tc2;
            const float2 g = *reinterpret_cast<const float2 *>(&raw.gate[r][ch]);
            const float2 k = bf2(*reinterpret_cast<const uint32_t *>(&raw.k[r][ch]));
            const float ax = ex2(chunk::floor_gate(g.x)), ay = ex2(chunk::floor_gate(g.y));
            t.s[j][0] = ax * (t.s[j][0] - k.x * n0); t.s[j][1] = ay * (t.s[j][1] - k.y * n0);
            t.s[j][2] = ax * (t.s[j][2] - k.x * n1); t.s[j][3] = ay * (t.s[j][3] - k.y * n1);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (8 * j + tc2 + (p & 1) == r) y[j][p] = t.inv * (p < 2 ? u0 : u1);
    }
    t.bound = 2.f * kLimit;
}

// Scale of a step's right-hand factors of largest element `nmax` that are added to the tile:
// the tile's own, or the tile comes down to theirs.  `ratio` is what its elements still have
// to be multiplied by; `grow` bounds what is added, without the scale.
__device__ __forceinline__ float join_scale(Tile &t, float nmax, float grow) {
    nmax = fmaxf(nmax, 0x1p-80f);
    // the tile has faded, or its bound is stale: 2^-8 leaves the largest factor its 11 bits, and six
    // octaves below it theirs
    if (chunk::uniform(nmax * t.c < 0x1p-8f)) t.renew();
    const float cn = scale_for(nmax, kTop);
    float ratio = 1.f;
    if (cn < t.c || t.bound == 0.f) {
        ratio = cn * t.inv;
        t.c = cn;
    }
    t.bound = t.bound * ratio + grow * t.c;
    return ratio;
}

// The tile as an operand, kept as the state at the slot's start.
__device__ __forceinline__ void store_tile(char *ckpt, const Tile &t, int tile, int lane) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        const float(&x)[4] = t.s[2 * kk], (&y)[4] = t.s[2 * kk + 1];
        reinterpret_cast<uint4 *>(ckpt)[(tile * 8 + kk) * 32 + lane] =
            make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(y[0], y[1]),
                       pack_f16(y[2], y[3]));
    }
}

// A [16 dv, 16 token] accumulator pair as the slot's FP16 block of a step and tile: a lane's
// words are (row lane / 4, tokens 2 (lane % 4), + 1), the row 8 below, and the same of tokens
// 8 - 15.  Returns the scale.
__device__ __forceinline__ float store_block(char *rows, const float (&x)[2][4], float largest,
                                             int block, int lane) {
    const float s = scale_for(fmaxf(largest, 1e-30f), kTop);
    reinterpret_cast<uint4 *>(rows)[block * 32 + lane] =
        make_uint4(pack_f16(x[0][0] * s, x[0][1] * s), pack_f16(x[0][2] * s, x[0][3] * s),
                   pack_f16(x[1][0] * s, x[1][1] * s), pack_f16(x[1][2] * s, x[1][3] * s));
    return s;
}

}  // namespace fast
}  // namespace kda
