// Matrix product with its epilogue for a few rows (decoding), the copy of rows onto 16-byte
// boundaries, and the first step of the backward pass.
#include <type_traits>

#include "kda_linear.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace linear {
namespace {

// y [M, N], M <= 8 MT.  Bound by memory: every weight is read once, straight from memory into the
// left operands of mma.sync (16 rows of the weight a CTA, the contraction cut over its eight warps);
// the few rows of x are the right operands.  Which k an operand's places stand for does not matter
// as long as both agree, so a lane takes 16 consecutive bytes of its row: four of them are two
// products' operands.  The tensor-memory path would move 128 rows of x for these few: 2048 x 8192 takes
// 5.1 us for 4 rows with the weight in L2, 8.6 for 16, and 15 there; 8192 x 2048 11.1 for 16, and 12.8.
constexpr int kWarps = 8, kAhead = 4;

template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    if (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The warps' sums of 16 weight rows from n0 on, [warp][MT][lane][register of the fragment], and the epilogue.
template <typename T, int MT>
__device__ __forceinline__ void finish(const GemmArgs &a, const float (*red)[MT][32][4], int n0) {
    // thread: one of 16 weight rows, one of 8 MT rows of x
    for (int e = threadIdx.x; e < 128 * MT; e += 32 * kWarps) {
        const int r = e & 15, m = e >> 4, t = m >> 3, n = n0 + r;
        // row r, column m % 8 of the 16 x 8 block: lane and register of the fragment
        const int l = (r & 7) * 4 + ((m & 7) >> 1), i = (r >> 3) * 2 + (m & 1);
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += red[w][t][l][i];
        if (m >= a.M || n >= a.N || !in_bounds(a.dbg, (size_t)m * a.N + n, (size_t)a.M * a.N, DBG_STORE)) continue;
        if (a.bias) v += as_f32(((const T *)a.bias)[n]);
        if (a.pre) ((T *)a.pre)[m * a.ldp + n] = from_f32<T>(v);
        v = activate(v, a.act);
        if (a.residual) v += as_f32(((const T *)a.residual)[m * a.ldr + n]);
        ((T *)a.y)[m * a.ldy + n] = from_f32<T>(v);
    }
}

template <typename T, int MT>
__global__ void __launch_bounds__(32 * kWarps) kda_linear_small_kernel(const GemmArgs a) {
    wait_for_previous();
    __shared__ float red[kWarps][MT][32][4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
    const int n0 = blockIdx.x * 16;
    const T *W = (const T *)a.B, *x = (const T *)a.A;
    float acc[MT][4] = {};
    const uint4 none = make_uint4(0, 0, 0, 0);
    // chunks of 32 k: chunk warp, warp + 8, ...
    const int chunks = (a.K + 31) / 32;
    for (int c0 = warp; c0 < chunks; c0 += kWarps * kAhead) {
        uint4 w[kAhead][2], b[kAhead][MT];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = (c0 + i * kWarps) * 32 + quad * 8;
            const bool in = k < a.K;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = n0 + row + 8 * h;
                w[i][h] = in && n < a.N && in_bounds(a.dbg, (size_t)n * a.K + k + 7, (size_t)a.N * a.K, DBG_LOAD)
                              ? *(const uint4 *)(W + (size_t)n * a.ldb + k) : none;
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int m = row + 8 * t;
                b[i][t] = in && m < a.M && in_bounds(a.dbg, (size_t)m * a.K + k + 7, (size_t)a.M * a.K, DBG_LOAD)
                              ? *(const uint4 *)(x + (size_t)m * a.lda + k) : none;
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                mma<T>(acc[t], w[i][0].x, w[i][1].x, w[i][0].y, w[i][1].y, b[i][t].x, b[i][t].y);
                mma<T>(acc[t], w[i][0].z, w[i][1].z, w[i][0].w, w[i][1].w, b[i][t].z, b[i][t].w);
            }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) *(float4 *)red[warp][t][lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    finish<T, MT>(a, red, n0);
}

// The same for a long contraction of few columns, where one CTA a multiprocessor has to keep memory busy: a
// warp of its own asks for whole rows of 1024 k several chunks ahead, also those of the CTA's next 16
// (one copy a row), and the rows of x beside them; eight warps take them from shared memory.  What
// lies in rows that are not there (behind N, behind M) becomes results that nobody takes.
constexpr int kChunk = 1024, kPitch = 2 * kChunk + 64;  // (64: eight lanes' banks are all different)

template <int MT> struct Long {
    static constexpr int kStage = (16 + 8 * MT) * kPitch, kStages = 4 / MT + (MT > 1);
    char raw[kStages][kStage];
    float red[kWarps][MT][32][4];
    uint64_t full[kStages], empty[kStages];
    uint32_t broken;
};

__device__ __forceinline__ void copy_row(void *to, const void *from, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_u32(to)),
                 "l"(from), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void sync_products() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

template <typename T, int MT>
__global__ void __launch_bounds__(32 * kWarps + 32, 1) kda_linear_long_kernel(const GemmArgs a) {
    wait_for_previous();
    using S = Long<MT>;
    extern __shared__ __align__(128) char smem[];
    S &s = *reinterpret_cast<S *>(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const T *W = (const T *)a.B, *x = (const T *)a.A;
    const int tiles = (a.N + 15) / 16, chunks = (a.K + kChunk - 1) / kChunk;
    volatile uint32_t *broken = &s.broken;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            tc::mbar_init(s.full + i, 1);
            tc::mbar_init(s.empty + i, kWarps);
        }
        *broken = 0;
        tc::fence_proxy_async_smem();
    }
    __syncthreads();
    auto wait = [&](uint64_t *bar, uint32_t parity) {  // (the lanes of a warp agree)
        const bool mine = !*broken && tc::mbar_wait(bar, parity, wait_polls(a.give_up));
        if (__all_sync(0xffffffffu, mine)) return true;
        *broken = 1;
        dbg_flag(a.dbg, true, DBG_WAIT);
        return false;
    };
    int n = 0;  // chunks so far
    if (warp == kWarps) {
        bool ok = true;
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            const int row = 16 * tile + lane, m = lane - 16;
            const bool mine = lane < 16 ? row < a.N && in_bounds(a.dbg, (size_t)row, (size_t)a.N, DBG_LOAD)
                                        : m < a.M && in_bounds(a.dbg, (size_t)m, (size_t)a.M, DBG_LOAD);
            const int there = __popc(__ballot_sync(0xffffffffu, mine));
            for (int c = 0; c < chunks; ++c, ++n) {
                const int st = n % S::kStages, k = c * kChunk;
                if (n >= S::kStages && !(ok = wait(s.empty + st, (n / S::kStages - 1) & 1))) break;
                const uint32_t bytes = min(kChunk, a.K - k) * 2;
                if (lane == 0) tc::mbar_arrive_expect_tx(s.full + st, there * bytes);
                __syncwarp();
                char *to = s.raw[st] + lane * kPitch;
                if (mine) copy_row(to, lane < 16 ? W + (size_t)row * a.ldb + k : x + (size_t)m * a.lda + k, bytes, s.full + st);
                __syncwarp();
            }
        }
        // every copy has landed before the CTA ends
        for (int i = max(0, n - S::kStages); i < n; ++i)
            tc::mbar_wait(s.full + i % S::kStages, (i / S::kStages) & 1, kWaitPolls);
        return;
    }
    const int row = lane >> 2, quad = lane & 3;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int n0 = 16 * tile;
        float acc[MT][4] = {};
        bool ok = true;
        for (int c = 0; c < chunks; ++c, ++n) {
            const int st = n % S::kStages, left = a.K - c * kChunk;
            ok = wait(s.full + st, (n / S::kStages) & 1) && ok;
            const char *at = s.raw[st] + row * kPitch + quad * 16;
#pragma unroll
            for (int i = 0; i < kChunk / 32 / kWarps; ++i) {
                const int k = (warp + kWarps * i) * 32;
                if (k >= left) break;
                const bool in = k + quad * 8 < left;
                uint4 w[2], b[MT];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[h] = in ? *(const uint4 *)(at + 8 * h * kPitch + 2 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    b[t] = in ? *(const uint4 *)(at + (16 + 8 * t) * kPitch + 2 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    mma<T>(acc[t], w[0].x, w[1].x, w[0].y, w[1].y, b[t].x, b[t].y);
                    mma<T>(acc[t], w[0].z, w[1].z, w[0].w, w[1].w, b[t].z, b[t].w);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(s.empty + st);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (!ok) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = __int_as_float(0x7fc00000);
            *(float4 *)s.red[warp][t][lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        }
        sync_products();
        finish<T, MT>(a, s.red, n0);
        sync_products();
    }
}

// Rows copied, eight elements a thread, up to two tensors in one launch.  A thread reads the 4-byte words
// that its elements lie in and shifts them by one where they begin in the middle of one (a word never
// ends outside the allocation that one of its bytes is in).
__global__ void __launch_bounds__(256) kda_linear_copy_kernel(const CopyArgs a0, const CopyArgs a1, unsigned first) {
    wait_for_previous();
    const CopyArgs &a = blockIdx.x < first ? a0 : a1;
    const int per = (a.width + 7) / 8;
    const long long i = (long long)(blockIdx.x - (blockIdx.x < first ? 0 : first)) * 256 + threadIdx.x, r = i / per;
    const int c = (int)(i - r * per) * 8, left = a.width - c;
    if (r >= a.rows || !in_bounds(a.dbg, (size_t)r, (size_t)a.rows, DBG_LOAD)) return;
    const uintptr_t at = (uintptr_t)((const uint16_t *)a.src + r * a.lds + c);
    const int s = at & 2 ? 1 : 0;  // elements of the first word in front of ours
    const uint32_t *f = (const uint32_t *)(at & ~(uintptr_t)3);
    uint32_t w[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = 2 * j - s < left && (j < 4 || s) ? f[j] : 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = __funnelshift_r(w[j], w[j + 1], 16 * s);
        if (2 * j + 1 >= left) w[j] &= 2 * j < left ? 0xffffu : 0u;
    }
    if (in_bounds(a.dbg, (size_t)(r * a.ldd + c + 7), (size_t)(a.rows * a.ldd), DBG_STORE))
        *(uint4 *)((uint16_t *)a.dst + r * a.ldd + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// dpre and the sums of its columns.  dpre is rounded to 16 bits because the products that read it take 16-bit
// operands; its sums take it as it is.  A warp has 32 V neighbouring columns of every eighth row of its
// CTA's part; the CTAs' sums are joined in order by a second kernel.  Bound by memory: 8192 x 8192 with
// gelu 77 us, 5.2 TB/s.
template <typename T, int V>
__global__ void __launch_bounds__(256) kda_linear_dact_kernel(const DActArgs a, int rows_each) {
    wait_for_previous();
    __shared__ float red[8][32 * V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockIdx.x * 32 * V + lane * V;
    const long long m0 = (long long)blockIdx.y * rows_each, m1 = min((long long)a.M, m0 + rows_each);
    float sum[V] = {};
    if (n < a.N) {
#pragma unroll 4
        for (long long m = m0 + warp; m < m1; m += 8) {
            if (!in_bounds(a.dbg, (size_t)m, (size_t)a.M, DBG_LOAD)) break;
            const auto dy = *(const Vec<T, V> *)((const T *)a.dy + m * a.lddy + n);
            Vec<T, V> p, d;
            if (a.act != ACT_NONE) p = *(const Vec<T, V> *)((const T *)a.pre + m * a.ldp + n);
            if constexpr (V == 1) {
                const float g = a.act != ACT_NONE ? dy[0] * slope(twice(p[0]), a.act).x : dy[0];
                sum[0] += g;
                d.v[0] = from_f32<T>(g);
            } else {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    float2 g = dy.two(i);
                    if (a.act != ACT_NONE) g = mul2(g, slope(p.two(i), a.act));
                    const float2 t = add2(make_float2(sum[i], sum[i + 1]), g);
                    sum[i] = t.x;
                    sum[i + 1] = t.y;
                    d.put(i, g);
                }
            }
            if (a.dpre && in_bounds(a.dbg, (size_t)(m * a.ldd + n + V - 1), (size_t)((a.M - 1) * a.ldd + a.N), DBG_STORE))
                *(Vec<T, V> *)((T *)a.dpre + m * a.ldd + n) = d;
        }
    }
    if (!a.dbias) return;
#pragma unroll
    for (int i = 0; i < V; ++i) red[warp][lane * V + i] = sum[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += red[w][i];
        const size_t at = (size_t)blockIdx.y * a.N + blockIdx.x * 32 * V + i;
        if (blockIdx.x * 32 * V + i < a.N && in_bounds(a.dbg, at, a.partial_floats, DBG_STORE)) a.partial[at] = s;
    }
}
template <typename T>
__global__ void __launch_bounds__(256) kda_linear_dbias_kernel(const DActArgs a, int n) {
    wait_for_previous();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.N) return;
    float s = 0.f;
#pragma unroll 8
    for (int i = 0; i < n; ++i)
        if (in_bounds(a.dbg, (size_t)i * a.N + c, a.partial_floats, DBG_LOAD)) s += a.partial[(size_t)i * a.N + c];
    if (in_bounds(a.dbg, (size_t)c, (size_t)a.N, DBG_STORE)) ((T *)a.dbias)[c] = from_f32<T>(s);
}

template <typename T, int V> cudaError_t dact(const DActArgs &a, cudaStream_t stream) {
    const int parts = dact_partials(a.M, a.N), each = (a.M + parts - 1) / parts;
    cudaError_t e = launch_early(kda_linear_dact_kernel<T, V>,
                                 dim3((unsigned)((a.N + 32 * V - 1) / (32 * V)), (unsigned)parts), 256, 0,
                                 stream, a, each);
    if (e != cudaSuccess || !a.dbias) return e;
    return launch_early(kda_linear_dbias_kernel<T>, (unsigned)((a.N + 255) / 256), 256, 0, stream, a, parts);
}
template <typename T> cudaError_t dact(const DActArgs &a, cudaStream_t stream) {
    Boundary u(2, a.N);
    u.add(a.dy, a.lddy);
    u.add(a.pre, a.ldp);
    u.add(a.dpre, a.ldd);
    return u.unit == 16 ? dact<T, 8>(a, stream) : u.unit == 8 ? dact<T, 4>(a, stream)
           : u.unit == 4 ? dact<T, 2>(a, stream) : dact<T, 1>(a, stream);
}

template <typename T, int MT> cudaError_t few(const GemmArgs &a, cudaStream_t stream) {
    // rows x K x N, weights from memory, us, straight and through shared memory: 4 x 2048 x 2048 5.8 and
    // 4.3, 4 x 8192 x 2048 18.7 and 9.4, 4 x 4096 x 4096 10.7 and 9.2, 16 x 8192 x 2048 19.1 and 12.1; but 4 x
    // 512 x 512 1.8 and 2.5, 4 x 1024 x 4096 4.1 and 4.7, 4 x 2048 x 8192 7.9 and 9.4, 8 x 8192 x 8192 26 and 33
    const int tiles = (a.N + 15) / 16;
    if (tiles > 2 * kSMs || a.K < 2 * kChunk)
        return launch_early(kda_linear_small_kernel<T, MT>, (unsigned)tiles, 32 * kWarps, 0, stream, a);
    constexpr int kBytes = sizeof(Long<MT>);
    static_assert(kBytes <= 227 * 1024, "");
    static volatile int done[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = smem_limit_once(kda_linear_long_kernel<T, MT>, kBytes, dev, done);
    if (e != cudaSuccess) return e;
    return launch_early(kda_linear_long_kernel<T, MT>, (unsigned)(tiles < kSMs ? tiles : kSMs), 32 * kWarps + 32, kBytes,
                        stream, a);
}
template <typename T> cudaError_t small(const GemmArgs &a, cudaStream_t stream) {
    return a.M <= 8 ? few<T, 1>(a, stream) : few<T, 2>(a, stream);
}

}  // namespace
}  // namespace linear

// Parts of the rows, each with a row of column sums: enough CTAs for the card at 256 columns each.
int dact_partials(int M, int N) {
    const long long blocks = (N + 255) / 256, want = (4 * kSMs + blocks - 1) / blocks;
    const long long most = (M + 31) / 32;
    const long long n = want < most ? want : most;
    return (int)(n < 1 ? 1 : n);
}

cudaError_t launch_dact(const DActArgs &a, cudaStream_t stream) {
    return a.fp16 ? linear::dact<__half>(a, stream) : linear::dact<__nv_bfloat16>(a, stream);
}

cudaError_t launch_copy_rows(const CopyArgs &a, const CopyArgs *b, cudaStream_t stream) {
    auto blocks = [](const CopyArgs &x) { return (unsigned)((x.rows * ((x.width + 7) / 8) + 255) / 256); };
    const unsigned first = blocks(a);
    return launch_early(linear::kda_linear_copy_kernel, first + (b ? blocks(*b) : 0), 256, 0, stream, a, b ? *b : a, first);
}

cudaError_t launch_small_gemm(const GemmArgs &a, cudaStream_t stream) {
    return a.fp16 ? linear::small<__half>(a, stream) : linear::small<__nv_bfloat16>(a, stream);
}

}  // namespace kda
