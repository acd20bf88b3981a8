// Matrix product with its epilogue on the tensor cores: C = A B^T, y = act(C + bias) + residual.
//
// Persistent, by role: one warp asks for the operands' tiles (TMA, 128-byte swizzle, 64 of K a stage),
// one issues the products (tcgen05.mma, accumulators in tensor memory), eight take the accumulators out
// and finish them (four are not enough beside 2048 of K where a gelu is taken and two results are
// written: 254 us at 8192 x 2048 x 8192 where eight take 163).  There are two accumulators, so that a
// tile's products run while the one before it is finished.  Operands may lie either way round: contracted
// along their rows' direction (K-major, boxes of 64 k) or across it (MN-major, boxes of 64 columns x 64
// k), which is what the gradients need of the same tensors.
//
// Large products take pairs of CTAs on neighbouring multiprocessors (cta_group::2): a tile of 256 x 256,
// each CTA holding 128 rows of A, 128 of B's rows and 128 of the accumulator's, and the first one's
// thread issuing products that read both's shared memory.  Alone, a CTA's tile of 128 x 256 fetches and
// reads half as much again a product, and shared memory is what runs out.  Where the tiles of C are too
// few for the card, the contraction is cut into parts whose sums a second kernel joins, always in the
// same order.
//
// Bound by the tensor cores, and by the power limit where calls follow one another for a second or more (1.5
// GHz instead of 2.07): 32768 x 2048 x 8192 bf16 with silu 636 us, 1.73 PFLOP/s (the library's plain product
// 613), and 557 in a burst (549).  In bursts: 788 without pairs, 705 with copies and products issued under a
// test of the lane, which makes the compiler take every operand of theirs through a loop; 8192 x 2048 x 8192
// with gelu and a second result 162, its gradients 395 with the 80 of their first step (256 tiles are 3.4 rounds of 76
// pairs; with whole tiles in the last one too 449).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "kda_linear.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace linear {
namespace {

constexpr int BM = 128, BK = 64;
constexpr int kEpilogue = 8;               // warps that finish tiles, 32 columns at a time
constexpr int kThreads = 64 + 32 * kEpilogue;

// BN: columns of a tile.  PAIR: of two CTAs, each with half of the rows of A and of B.
template <int BN, bool PAIR> struct Cfg {
    static constexpr int kRowsB = PAIR ? BN / 2 : BN;  // of B in this CTA
    static constexpr int kA = BM * BK * 2, kB = kRowsB * BK * 2, kStage = kA + kB;
    static constexpr int kStages = 204800 / kStage < 6 ? 204800 / kStage : 6;
    static constexpr int kOut = kEpilogue * 2048;  // a [32 rows x 32 columns] box of each epilogue warp
    static constexpr int kBias = kEpilogue * (BN / 2) * 4;
    static constexpr int kBytes = 1024 + kStages * kStage + kOut + kBias + 256;
    static constexpr int kColumns = BN > 128 ? 512 : 2 * BN;  // of tensor memory: a power of two
};

struct Maps {
    CUtensorMap a, b, y, pre;
};

struct Params {
    int M, N, K, nt, tiles, splits, per;  // tiles across N; of C; parts of K, blocks of 64 of each
    int rows_a;      // of A in a copy
    int work, full;  // pieces of work; those from `full` on are halves of tiles
    const void *bias, *residual;
    void *y, *pre;
    long long ldr, ldy, ldp;
    int act;
    float *partial;  // [splits][M][ldw], or null
    size_t partial_floats;
    int ldw;
    bool tma_out;         // y and pre leave by TMA
    int unit_o, unit_r;   // bytes on whose boundaries their rows begin, and residual's
    unsigned *dbg;
    bool give_up;
};

// Shared-memory descriptor, 128-byte swizzle: K-major sbo = 1024 (eight rows); MN-major sbo = 1024
// (eight k), lbo = from 64 columns to the next.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return tc::smem_desc(addr, lbo, sbo) | (uint64_t)2 << 61;
}
// FP32 sums of 16-bit operands.
constexpr uint32_t idesc16(bool fp16, bool a_mn, bool b_mn, int m, int n) {
    return 1u << 4 | (fp16 ? 0u : 1u) << 7 | (fp16 ? 0u : 1u) << 10 | (uint32_t)a_mn << 15 |
           (uint32_t)b_mn << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}
template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (PAIR)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}
// Arrives on the barrier (of a pair: on both CTAs') when this thread's products so far are done.
template <bool PAIR> __device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                tc::smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        tc::mma_commit(bar);
}
// A pair's copies all report to the first CTA's barrier; `bar` is its address in the cluster then.
template <bool PAIR>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
template <bool PAIR> __device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t columns) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(slot)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tc::tmem_alloc(slot, columns);
    }
}
template <bool PAIR> __device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
    else
        tc::tmem_dealloc(at, columns);
}
// Bounded wait as tc::mbar_wait, with what the pair's other CTA did before it arrived.
__device__ __forceinline__ bool wait_pair(uint64_t *bar, uint32_t parity, uint32_t polls) {
    const uint32_t a = tc::smem_u32(bar);
    for (uint32_t i = 0; i < polls; ++i) {
        uint32_t done;
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done)
            : "r"(a), "r"(parity)
            : "memory");
        if (done) return true;
    }
    return false;
}
// Arrives on the first CTA's barrier.
__device__ __forceinline__ void arrive_first(uint64_t *bar) {
    asm volatile(
        "{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, 0;\n"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(tc::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ uint32_t in_first(uint64_t *bar) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(tc::smem_u32(bar)));
    return a;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void store_2d(const CUtensorMap *map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]),
          "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}

struct Tile {
    int m, n, cols, kb, ke;  // first row and column, columns, blocks of K
};
// Tiles go down 16 rows of tiles before the next column, so that those at work at one time share
// both operands' tiles in L2.
__device__ __forceinline__ Tile tile_of(const Params &p, int i, int rows_each, int BN) {
    Tile t;
    const bool half = i >= p.full, right = half && (i - p.full & 1);
    if (half) i = p.full + (i - p.full) / 2;
    const int s = i / p.tiles, j = i - s * p.tiles, mt = p.tiles / p.nt;
    const int group = j / (16 * p.nt), rows = min(16, mt - group * 16), r = j - group * 16 * p.nt;
    t.m = (group * 16 + r % rows) * rows_each;
    t.n = r / rows * BN + (right ? BN / 2 : 0);
    t.cols = half ? BN / 2 : BN;
    t.kb = s * p.per;
    t.ke = min(t.kb + p.per, (p.K + BK - 1) / BK);
    return t;
}

template <int ACT> __device__ __forceinline__ void activate_as(float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 y = activate<ACT>(make_float2(v[j], v[j + 1]));
        v[j] = y.x;
        v[j + 1] = y.y;
    }
}
__device__ __forceinline__ void activate_all(float (&v)[32], int act) {
    if (act == ACT_SILU)
        activate_as<ACT_SILU>(v);
    else if (act == ACT_GELU)
        activate_as<ACT_GELU>(v);
    else if (act == ACT_RELU)
        activate_as<ACT_RELU>(v);
}

// Where 16 bytes (chunk q) of row r are in a box of 32 rows of 64 bytes, swizzled as the tensor maps of
// the results are.
__device__ __forceinline__ int spot(int r, int q) { return r * 64 + ((q ^ (r >> 1 & 3)) << 4); }

// A box from or to rows that begin on boundaries of a word W: neighbouring lanes have neighbouring words;
// words that the last column ends in go by elements.
template <typename W> struct Rows {
    static constexpr int kWords = 64 / sizeof(W), kStep = 32 / kWords, kEach = sizeof(W) / 2;
    int row, byte, left;  // this lane's first row, place in it, and elements from there to the last column
    int N;
    unsigned *dbg;
    __device__ __forceinline__ Rows(int n, int N, int lane, unsigned *dbg)
        : row(lane / kWords), byte(lane % kWords * (int)sizeof(W)), left(N - n - byte / 2), N(N), dbg(dbg) {}
    // Whether this lane's elements of row r, from column n on, are the tensor's.
    __device__ __forceinline__ bool ok(long long ld, int r, int n, int M, unsigned bit) const {
        return left <= 0 || in_bounds(dbg, (size_t)r * ld + n + byte / 2 + min(left, kEach) - 1, (size_t)(M - 1) * ld + N, bit);
    }
    __device__ __forceinline__ void in(char *box, const void *base, long long ld, int m, int n, int M) const {
        const uint16_t *at = (const uint16_t *)base + (size_t)(m + row) * ld + n + byte / 2;
        const int rows = min(32, M - m);
        constexpr int kBatch = 32 / kStep < 16 ? 32 / kStep : 16;  // each waits for memory once
#pragma unroll
        for (int b = 0; b < 32 / kStep; b += kBatch) {
            W x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = row + (b + i) * kStep;
                const uint16_t *f = at + (size_t)(b + i) * kStep * ld;
                x[i] = W{};
                if (r < rows && !ok(ld, m + r, n, M, DBG_LOAD)) continue;
                if (r < rows && left >= kEach) {
                    x[i] = *(const W *)f;
                } else if (r < rows && left > 0) {
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        if (e < left) ((uint16_t *)&x[i])[e] = f[e];
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                *(W *)(box + spot(row + (b + i) * kStep, byte >> 4) + (byte & 15)) = x[i];
        }
    }
    __device__ __forceinline__ void out(const char *box, void *base, long long ld, int m, int n, int M) const {
        uint16_t *to = (uint16_t *)base + (size_t)(m + row) * ld + n + byte / 2;
        const int rows = min(32, M - m);
#pragma unroll 8
        for (int r = row; r < rows; r += kStep, to += kStep * ld) {
            const W x = *(const W *)(box + spot(r, byte >> 4) + (byte & 15));
            if (!ok(ld, m + r, n, M, DBG_STORE)) continue;
            if (left >= kEach) {
                *(W *)to = x;
            } else {
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (e < left) to[e] = ((const uint16_t *)&x)[e];
            }
        }
    }
};
__device__ __forceinline__ void box_in(char *box, const void *base, long long ld, int m, int n, int M, int N, int lane,
                                       int unit, unsigned *dbg) {
    if (unit == 16)
        Rows<uint4>(n, N, lane, dbg).in(box, base, ld, m, n, M);
    else if (unit == 8)
        Rows<uint2>(n, N, lane, dbg).in(box, base, ld, m, n, M);
    else if (unit == 4)
        Rows<uint32_t>(n, N, lane, dbg).in(box, base, ld, m, n, M);
    else
        Rows<uint16_t>(n, N, lane, dbg).in(box, base, ld, m, n, M);
}
__device__ __forceinline__ void box_out(const char *box, void *base, long long ld, int m, int n, int M, int N, int lane,
                                        int unit, unsigned *dbg) {
    if (unit == 16)
        Rows<uint4>(n, N, lane, dbg).out(box, base, ld, m, n, M);
    else if (unit == 8)
        Rows<uint2>(n, N, lane, dbg).out(box, base, ld, m, n, M);
    else if (unit == 4)
        Rows<uint32_t>(n, N, lane, dbg).out(box, base, ld, m, n, M);
    else
        Rows<uint16_t>(n, N, lane, dbg).out(box, base, ld, m, n, M);
}

template <typename T, bool A_MN, bool B_MN, int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    kda_linear_kernel(const __grid_constant__ Maps maps, const Params p) {
    wait_for_previous();
    using C = Cfg<BN, PAIR>;
    constexpr int kRows = PAIR ? 2 * BM : BM;  // of a tile
    extern __shared__ char raw[];
    char *base = (char *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    char *out = base + C::kStages * C::kStage;
    float *bias = (float *)(out + C::kOut);
    uint64_t *full = (uint64_t *)((char *)bias + C::kBias), *empty = full + C::kStages;
    uint64_t *done = empty + C::kStages, *taken = done + 2;
    uint32_t *slot = (uint32_t *)(taken + 2);
    volatile uint32_t *broken = slot + 1;
    // (said to be the same in all lanes: in code that might diverge, every operand of an asynchronous
    // instruction goes through a loop over the lanes, and a stage took 810 cycles instead of 512)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int work = p.work;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    const int first = PAIR ? (int)blockIdx.x / 2 : (int)blockIdx.x, step = PAIR ? (int)gridDim.x / 2 : (int)gridDim.x;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(full + i, 1);
            tc::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(done + i, 1);
            tc::mbar_init(taken + i, PAIR ? 2 * kEpilogue : kEpilogue);
        }
        *broken = 0;
    }
    if (warp == 1) tmem_alloc<PAIR>(slot, C::kColumns);
    __syncthreads();
    if (PAIR) cluster_sync();  // both CTAs' barriers are there
    tc::fence_after_sync();
    const uint32_t tmem = *slot;
    // A wait that gives up ends this CTA's copies and products; the other warps learn of it here, and the
    // finishing ones write NaN to the tile at hand and to all that are left.
    const uint32_t polls = wait_polls(p.give_up);
    // (the lanes of a warp agree: one of them may see that another warp gave up while the others see the barrier,
    // and what follows is for whole warps)
    auto poll = [&](uint64_t *bar, uint32_t parity, uint32_t n) {
        return PAIR ? wait_pair(bar, parity, n) : tc::mbar_wait(bar, parity, n);
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, !*broken && poll(bar, parity, polls))) return true;
        *broken = 1;
        dbg_flag(p.dbg, true, DBG_WAIT);
        return false;
    };
    // The same for the warps that leave their loop at the first wait that fails, and so never wait for a phase
    // behind one that they have not seen: most waits are over at the first poll, without a look at `broken`.
    auto wait_in_order = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, poll(bar, parity, min(polls, 1u))) || wait(bar, parity);
    };
    if (warp == 0) {
        int n = 0;  // stages filled so far
        const uint32_t bars = PAIR ? in_first(full) : tc::smem_u32(full);
        bool ok = true;
        for (int i = first; i < work && ok; i += step) {
            const Tile t = tile_of(p, i, kRows, BN);
            const int rows = PAIR ? t.cols / 2 : C::kRowsB, m = t.m + rank * BM, nn = t.n + rank * rows;
            for (int kb = t.kb; kb < t.ke; ++kb, ++n) {
                const int st = n % C::kStages;
                if (n >= C::kStages && !(ok = wait_in_order(empty + st, (n / C::kStages - 1) & 1))) break;
                if (tc::elect_one()) {
                    const uint32_t a = tc::smem_u32(base + st * C::kStage), b = a + C::kA;
                    // (a pair's first CTA waits for both's bytes)
                    if (!PAIR || rank == 0) tc::mbar_arrive_expect_tx(full + st, (PAIR ? 2 : 1) * (p.rows_a + rows) * BK * 2);
                    if (A_MN) {
#pragma unroll
                        for (int x = 0; x < BM / 64; ++x)
                            load_2d<PAIR>(a + x * 8192, &maps.a, m + 64 * x, kb * BK, bars + 8 * st);
                    } else {
                        load_2d<PAIR>(a, &maps.a, kb * BK, m, bars + 8 * st);
                    }
                    if (B_MN || PAIR) {
#pragma unroll
                        for (int x = 0; x < C::kRowsB / 64; ++x)
                            if (64 * x < rows)
                                load_2d<PAIR>(b + x * 8192, &maps.b, B_MN ? nn + 64 * x : kb * BK,
                                              B_MN ? kb * BK : nn + 64 * x, bars + 8 * st);
                    } else {
                        load_2d<PAIR>(b, &maps.b, kb * BK, nn, bars + 8 * st);
                    }
                }
                __syncwarp();
            }
        }
        // every copy has landed before the CTA ends (a pair's: before its first CTA does)
        for (int s = max(0, n - C::kStages); s < n && rank == 0; ++s)
            tc::mbar_wait(full + s % C::kStages, (s / C::kStages) & 1, kWaitPolls);
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr bool fp16 = std::is_same<T, __half>::value;
            constexpr uint32_t whole = idesc16(fp16, A_MN, B_MN, kRows, BN), half = idesc16(fp16, A_MN, B_MN, kRows, BN / 2);
            constexpr uint32_t kStepA = A_MN ? 2048 : 32, kStepB = B_MN ? 2048 : 32;  // 16 of K
            int n = 0, c = 0;
            bool ok = true;
            for (int i = first; i < work && ok; i += step, ++c) {
                const Tile t = tile_of(p, i, kRows, BN);
                if (c >= 2 && !wait_in_order(taken + (c & 1), (c / 2 - 1) & 1)) break;
                tc::fence_after_sync();
                const uint32_t d = tmem + (c & 1) * BN, idesc = PAIR && t.cols < BN ? half : whole;
                for (int kb = t.kb; kb < t.ke; ++kb, ++n) {
                    const int st = n % C::kStages;
                    if (!(ok = wait_in_order(full + st, (n / C::kStages) & 1))) break;
                    tc::fence_after_sync();
                    const uint32_t a = tc::smem_u32(base + st * C::kStage), b = a + C::kA;
                    if (tc::elect_one()) {
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            mma_f16<PAIR>(d, desc128(a + k * kStepA, A_MN ? 8192 : 16, 1024),
                                          desc128(b + k * kStepB, B_MN ? 8192 : 16, 1024), idesc,
                                          kb > t.kb || k > 0);
                        commit<PAIR>(empty + st);
                        if (kb + 1 == t.ke) commit<PAIR>(done + (c & 1));
                    }
                    __syncwarp();
                }
            }
            // the last products are done with the stages before the CTA ends
            if (n > 0) tc::mbar_wait(empty + (n - 1) % C::kStages, ((n - 1) / C::kStages) & 1, kWaitPolls);
        }
    } else {
        // a warp reads its own 32 lanes of tensor memory, and takes half of a tile's columns
        const int e = warp - 2, quarter = warp & 3;
        char *box = out + e * 2048;
        float *bs = bias + e * (BN / 2);
        int c = 0;
        auto begin = [&] {  // the box may be written
            if (p.tma_out) {
                if (lane == 0) tc::bulk_wait_read_all();
                __syncwarp();
            }
        };
        for (int i = first; i < work; i += step, ++c) {
            const Tile t = tile_of(p, i, kRows, BN);
            const int each = PAIR ? t.cols / 2 : BN / 2, c0 = e / 4 * each;
            const int m0 = t.m + rank * BM + 32 * quarter, n0 = t.n + c0, n1 = min(p.N - n0, each);
            auto addend = [&](int n) {
                begin();
                box_in(box, p.residual, p.ldr, m0, n0 + n, p.M, p.N, lane, p.unit_r, p.dbg);
                __syncwarp();
            };
            const bool early = p.residual && !p.pre && !p.partial && n1 > 0;
            if (!p.partial) {
                __syncwarp();
                for (int j = lane; j < BN / 2; j += 32)
                    bs[j] = p.bias && n0 + j < p.N && in_bounds(p.dbg, (size_t)(n0 + j), (size_t)p.N, DBG_LOAD)
                                ? as_f32(((const T *)p.bias)[n0 + j]) : 0.f;
                __syncwarp();
                if (early) addend(0);
            }
            const bool ok = wait(done + (c & 1), (c / 2) & 1);
            tc::fence_after_sync();
            const uint32_t d = tmem + (c & 1) * BN + c0 + ((uint32_t)quarter << 21);
            int n = 0;
            do {
                float v[32];
                if (n1 > 0 && ok) {
                    tmem_ld32(d + n, v);
                    tc::tmem_wait_ld();
                }
                if (n + 32 >= n1) {  // the accumulator may be written again
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR)
                            arrive_first(taken + (c & 1));
                        else
                            tc::mbar_arrive(taken + (c & 1));
                    }
                    if (n1 <= 0) break;
                }
                if (!ok) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __int_as_float(0x7fc00000);
                }
                if (p.partial) {
                    const int m = m0 + lane;
                    if (m < p.M) {
                        const size_t at = ((size_t)(i / p.tiles) * p.M + m) * p.ldw + n0 + n;
                        float *to = p.partial + at;
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            if (n0 + n + j < p.ldw && in_bounds(p.dbg, at + j + 3, p.partial_floats, DBG_STORE))
                                *(float4 *)(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    }
                    continue;
                }
                if (p.bias) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 b = *(const float4 *)(bs + n + j);
                        v[j] += b.x; v[j + 1] += b.y; v[j + 2] += b.z; v[j + 3] += b.w;
                    }
                }
                // a box of 32 rows x 32 columns at a time: pre, then y
                auto put = [&](bool add) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 *at = (uint4 *)(box + spot(lane, q));
                        if (add) {
                            const uint4 r = *at;
                            const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float2 f = unpack<T>(rr[x]);
                                v[8 * q + 2 * x] += f.x;
                                v[8 * q + 2 * x + 1] += f.y;
                            }
                        }
                        *at = make_uint4(pack<T>(v[8 * q], v[8 * q + 1]), pack<T>(v[8 * q + 2], v[8 * q + 3]),
                                         pack<T>(v[8 * q + 4], v[8 * q + 5]), pack<T>(v[8 * q + 6], v[8 * q + 7]));
                    }
                };
                auto leave = [&](const CUtensorMap *map, void *to, long long ld) {
                    if (p.tma_out) {
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && m0 < p.M) {
                            store_2d(map, tc::smem_u32(box), n0 + n, m0);
                            tc::bulk_commit_group();
                        }
                    } else {
                        __syncwarp();
                        box_out(box, to, ld, m0, n0 + n, p.M, p.N, lane, p.unit_o, p.dbg);
                        __syncwarp();
                    }
                };
                if (p.pre) {
                    begin();
                    put(false);
                    leave(&maps.pre, p.pre, p.ldp);
                }
                activate_all(v, p.act);
                if (!p.residual)
                    begin();
                else if (!early || n > 0)
                    addend(n);
                put(p.residual);
                leave(&maps.y, p.y, p.ldy);
            } while ((n += 32) < n1);
        }
        if (lane == 0) tc::bulk_wait_all();
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (PAIR) cluster_sync();  // neither CTA's shared memory is wanted any more
    tc::fence_after_sync();
    if (warp == 1) tmem_free<PAIR>(tmem, C::kColumns);
}

// The parts of the contraction joined, with the epilogue: a thread has four columns of a row.
template <typename T>
__global__ void __launch_bounds__(256) kda_linear_join_kernel(const Params p) {
    wait_for_previous();
    const int quads = p.ldw / 4;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long m = i / quads;
    const int n = (int)(i - m * quads) * 4;
    if (m >= p.M) return;
    const float *at = p.partial + m * p.ldw + n;
    float v[4] = {};
    for (int s = 0; s < p.splits; ++s) {
        const float *part = at + (size_t)s * p.M * p.ldw;
        if (!in_bounds(p.dbg, (size_t)(part - p.partial) + 3, p.partial_floats, DBG_LOAD)) continue;
        const float4 x = *(const float4 *)part;
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= p.N || !in_bounds(p.dbg, (size_t)m * p.N + n + j, (size_t)p.M * p.N, DBG_STORE)) break;
        const float x = v[j] + (p.bias ? as_f32(((const T *)p.bias)[n + j]) : 0.f);
        if (p.pre) ((T *)p.pre)[m * p.ldp + n + j] = from_f32<T>(x);
        float y = activate(x, p.act);
        if (p.residual) y += as_f32(((const T *)p.residual)[m * p.ldr + n + j]);
        ((T *)p.y)[m * p.ldy + n + j] = from_f32<T>(y);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

cudaError_t encode(CUtensorMap *m, bool fp16, const void *base, long long cols, long long rows,
                   long long ld, int box_cols, int box_rows, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                               cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, one[2] = {1, 1};
    auto fill = [&] {
        return g_encode(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                        const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = fill();
    int dev = 0;
    // a thread that has made no call of the runtime's before (autograd runs backward on such) has no
    // current context, which this call of the driver's needs; setting the device makes one current
    if (r != CUDA_SUCCESS && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = fill();
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Columns of a tile, pairs or not, and parts of the contraction.
struct Plan {
    int bn, tiles, splits, per, ldw;
    bool pair;
};
Plan plan_of(int M, int N, int K) {
    Plan q;
    auto tiles = [&](int bm, int bn) { return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
    // pairs of CTAs: where there is a tile for each, or where a long contraction outweighs the 3 us that
    // they start later (alone and in pairs, us: 8192 x 2048 x 2048, 256 tiles, 60 and 44; 2560 x 2048 x
    // 4096, 80 tiles, 48 and 42; 2048 x 1280 x 4096, 40 tiles, 26.5 and 25.4; 1536 x 2048 x 2048, 48
    // tiles, 16.0 and 16.7; 32 x 8192 x 8192, 32 tiles, 40 and 42)
    q.pair = tiles(256, 256) >= (K >= 4096 ? 40 : kSMs / 2);
    q.bn = 256;
    if (!q.pair) {
        // the width whose rounds of tiles take least: a stage's products take BN / 4 of 64 cycles, its
        // start and the tile's ends some 48 columns' worth (2021 x 1540 x 1111: 192 columns take one
        // round of 144 tiles, 128 two of 208)
        long long best = -1;
        for (int bn = 64; bn <= 256; bn += 64) {
            const long long cost = (tiles(BM, bn) + kSMs - 1) / kSMs * (bn + 48);
            if (best < 0 || cost < best || (cost == best && tiles(BM, bn) * 2 <= kSMs)) {
                best = cost;
                q.bn = bn;
            }
        }
        if (tiles(BM, q.bn) * 2 <= kSMs) q.bn = N > 64 ? 128 : 64;  // the contraction is cut anyway
    }
    q.tiles = (int)tiles(q.pair ? 2 * BM : BM, q.bn);
    const int blocks = (K + BK - 1) / BK;
    int splits = !q.pair && q.tiles * 2 <= kSMs ? kSMs / q.tiles : 1;
    if (splits > blocks / 4) splits = blocks / 4;  // four blocks of 64 at least
    if (splits > 16) splits = 16;
    if (splits < 1) splits = 1;
    q.per = (blocks + splits - 1) / splits;
    q.splits = blocks ? (blocks + q.per - 1) / q.per : 1;
    q.ldw = (N + 3) / 4 * 4;
    return q;
}

template <typename T, bool A_MN, bool B_MN, int BN, bool PAIR>
cudaError_t launch(const Maps &maps, const Params &p, cudaStream_t stream) {
    auto kernel = kda_linear_kernel<T, A_MN, B_MN, BN, PAIR>;
    constexpr int kBytes = Cfg<BN, PAIR>::kBytes;
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = smem_limit_once(kernel, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    const int work = p.work;
    if (!PAIR) return launch_early(kernel, (unsigned)(work < kSMs ? work : kSMs), kThreads, kBytes, stream, maps, p);
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = 2;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)(work < kSMs / 2 ? work : kSMs / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}
template <typename T, bool A_MN, bool B_MN>
cudaError_t pick(const Plan &q, const Maps &maps, const Params &p, cudaStream_t stream) {
    if (q.pair) return launch<T, A_MN, B_MN, 256, true>(maps, p, stream);
    return q.bn == 256 ? launch<T, A_MN, B_MN, 256, false>(maps, p, stream)
           : q.bn == 192 ? launch<T, A_MN, B_MN, 192, false>(maps, p, stream)
           : q.bn == 128 ? launch<T, A_MN, B_MN, 128, false>(maps, p, stream)
                         : launch<T, A_MN, B_MN, 64, false>(maps, p, stream);
}
template <typename T> cudaError_t run(const GemmArgs &a, cudaStream_t stream) {
    const Plan q = plan_of(a.M, a.N, a.K);
    Maps maps;
    // what lies in shared memory behind the last row of a few becomes rows of the result that nobody takes
    // (17 rows, 2048 x 8192: 11.3 us with the weight in L2; zeros copied there cost 4.4 more)
    const int rows_a = !a.a_mn && a.M < BM ? (a.M + 7) / 8 * 8 : BM;
    cudaError_t e = a.a_mn ? encode(&maps.a, a.fp16, a.A, a.M, a.K, a.lda, 64, BK)
                           : encode(&maps.a, a.fp16, a.A, a.K, a.M, a.lda, BK, rows_a);
    if (e == cudaSuccess)
        e = a.b_mn ? encode(&maps.b, a.fp16, a.B, a.N, a.K, a.ldb, 64, BK)
                   : encode(&maps.b, a.fp16, a.B, a.K, a.N, a.ldb, BK, q.pair ? 64 : q.bn);
    if (e != cudaSuccess) return e;
    Params p = {};
    p.M = a.M; p.N = a.N; p.K = a.K;
    p.nt = (a.N + q.bn - 1) / q.bn;
    p.tiles = q.tiles; p.splits = q.splits; p.per = q.per;
    p.rows_a = rows_a;
    p.work = q.tiles * q.splits;
    p.full = p.work;
    // pairs share the last round out by halves of tiles where that leaves no second one
    const int rest = q.pair ? q.tiles % (kSMs / 2) : 0;
    if (rest * 2 <= kSMs / 2) {
        p.work += rest;
        p.full -= rest;
    }
    p.bias = a.bias; p.residual = a.residual; p.y = a.y; p.pre = a.pre;
    p.ldr = a.ldr; p.ldy = a.ldy; p.ldp = a.ldp;
    p.act = a.act;
    p.ldw = q.ldw;
    p.partial = q.splits > 1 ? a.partial : nullptr;
    p.partial_floats = a.partial_floats;
    p.dbg = a.dbg;
    p.give_up = a.give_up;
    Boundary o(2, 8), r(2, 8);
    o.add(a.y, a.ldy);
    o.add(a.pre, a.ldp);
    r.add(a.residual, a.ldr);
    p.unit_o = o.unit;
    p.unit_r = r.unit;
    p.tma_out = !p.partial && o.unit == 16;
    if (p.tma_out) {
        e = encode(&maps.y, a.fp16, a.y, a.N, a.M, a.ldy, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
        if (e == cudaSuccess && a.pre) e = encode(&maps.pre, a.fp16, a.pre, a.N, a.M, a.ldp, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
        if (e != cudaSuccess) return e;
    }
    e = a.a_mn ? pick<T, true, true>(q, maps, p, stream)
        : a.b_mn ? pick<T, false, true>(q, maps, p, stream) : pick<T, false, false>(q, maps, p, stream);
    if (e != cudaSuccess || !p.partial) return e;
    const long long quads = (long long)a.M * (q.ldw / 4);
    return launch_early(kda_linear_join_kernel<T>, (unsigned)((quads + 255) / 256), 256, 0, stream, p);
}

}  // namespace
}  // namespace linear

size_t gemm_partial_bytes(int M, int N, int K) {
    const linear::Plan q = linear::plan_of(M, N, K);
    return q.splits > 1 ? (size_t)q.splits * M * q.ldw * 4 : 0;
}

cudaError_t launch_gemm(const GemmArgs &a, cudaStream_t stream) {
    return a.fp16 ? linear::run<__half>(a, stream) : linear::run<__nv_bfloat16>(a, stream);
}

}  // namespace kda
