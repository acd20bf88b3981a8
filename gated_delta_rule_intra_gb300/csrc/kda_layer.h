// Internal launch interface of the short convolution, the selective scan and the matrix product
// with its epilogue.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "kda_ops.h"

namespace kda {

// Element types (as the layer norm's) and activations.
enum { TYPE_BF16 = NORM_BF16, TYPE_FP16 = NORM_FP16, TYPE_FP32 = NORM_FP32 };
enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2, ACT_RELU = 3 };

inline int esize(int dtype) { return dtype == TYPE_FP32 ? 4 : 2; }

// Tokens of a batch [B, T], or packed along T (B = 1) with cu_seqlens.
struct Tokens {
    int B, T, num_seqs;      // num_seqs = B without cu_seqlens
    const int *cu_seqlens;   // [num_seqs + 1] or null
    constexpr long long rows() const { return (long long)B * T; }
    // Pieces of `size` tokens, at most (find_piece() in kda_rows.cuh).
    constexpr long long pieces(int size) const {
        return cu_seqlens ? (long long)T / size + num_seqs
                          : (long long)B * (T > size ? (T + size - 1) / size : 1);
    }
};

struct ConvArgs {
    Tokens tok;
    const void *x, *weight, *bias;  // x [rows, D]; weight [D, W], bias [D] (null = 0) of wdtype
    void *y;
    const void *initial;            // [num_seqs, W - 1, D] of x's type, or null = zeros
    void *final;                    // the same, or null
    int D, W, dtype, wdtype, act;
    long long x_stride, y_stride, dy_stride, dx_stride;  // elements between rows
    // backward
    const void *dy;
    void *dx;
    const void *d_final;            // [num_seqs, W - 1, D] of x's type, or null
    void *d_initial;                // the same, or null
    float *dweight, *dbias;         // [D, W], [D]; both or none
    float *partial;                 // [partials][W + 1][D]
    int partials;
    size_t partial_floats;          // in the workspace, for the debug build's checks
    // single tokens
    void *state;                    // [num_states, W - 1, D]
    const int *state_indices;
    int N;
    long long num_states;
    unsigned *dbg;
};

cudaError_t launch_conv_fwd(const ConvArgs &a, cudaStream_t stream);
cudaError_t launch_conv_bwd(const ConvArgs &a, cudaStream_t stream);
cudaError_t launch_conv_step(const ConvArgs &a, cudaStream_t stream);
constexpr int kConvPiece = 96;  // tokens that a CTA of the backward takes at a time
int conv_partials(long long pieces, int D);

struct ScanArgs {
    Tokens tok;
    const void *u, *delta, *z, *B, *C;   // [rows, D] (z: or null), [rows, G, N], one type
    const float *A, *skip, *delta_bias;  // [D, N], [D] or null
    void *y;
    const float *initial;                // [num_seqs, D, N] or null = zeros
    float *final;                        // the same, or null
    float *saved;                        // states in front of every kScanTile / 2 tokens, or null
    float *open;                         // [rows, D rounded up to 4]: y before the gate, or null
    int D, N, G, dtype;
    bool softplus;
    long long u_stride, delta_stride, z_stride, B_stride, C_stride, y_stride;
    int segment;                         // tokens that one CTA walks, a multiple of kScanTile
    float *ends, *sums;                  // [segments][D][NP], [segments][D] (null: none)
    // backward
    const void *dy;
    void *du, *ddelta, *dz, *dB, *dC;    // dz null with z
    float *dA, *dskip, *ddelta_bias;     // dskip, ddelta_bias: null with skip, delta_bias
    const float *d_final;                // [num_seqs, D, N] or null = zeros
    float *d_initial;                    // the same, or null
    long long dy_stride, du_stride, ddelta_stride, dz_stride;
    float *part_bc, *part_A, *part_D;    // [blocks][rows][G][2 NP], [segments][D][NP], [..][2][D]
    // single tokens
    float *state;                        // [num_states, D, N]
    const int *state_indices;
    int requests;
    long long num_states;
    // for the debug build's checks: elements of `saved`, of `open`, of `ends` and `part_A`, of `sums`, ...
    size_t saved_floats, open_floats, segment_floats, sum_floats, part_D_floats, part_bc_floats;
    unsigned *dbg;
};

constexpr int kScanTile = 16, kScanMaxN = 64;
inline int scan_padded(int N) {  // NP: states of a channel, padded
    int np = 8;
    while (np < N) np *= 2;
    return np;
}
inline int scan_channels(int N) { return 1024 / scan_padded(N); }  // of a CTA
inline long long scan_blocks(int D, int N, int G) {               // CTAs side by side
    const int ch = scan_channels(N);
    return (long long)G * ((D / G + ch - 1) / ch);
}
int scan_segment(const Tokens &tok, int D, int N, int G, bool back);
cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t stream);
cudaError_t launch_scan_bwd(const ScanArgs &a, cudaStream_t stream);
cudaError_t launch_scan_step(const ScanArgs &a, cudaStream_t stream);

// C [M, N] = A B^T of 16-bit operands, FP32 sums.  A is [M, K] (or [K, M] with a_mn), B [N, K] (or
// [K, N] with b_mn); rows on 16-byte boundaries, ld elements apart.
struct GemmArgs {
    const void *A, *B;
    long long lda, ldb;
    bool a_mn, b_mn;
    int M, N, K;
    // y = act(C + bias) + residual, pre = C + bias, both of the operands' type; bias, residual and pre
    // may be null
    const void *bias, *residual;
    void *y, *pre;
    long long ldr, ldy, ldp;
    int act;
    bool fp16;
    float *partial;  // gemm_partial_bytes()
    size_t partial_floats;
    unsigned *dbg;
    bool give_up;  // debug build: its bounded waits give up at once
};
size_t gemm_partial_bytes(int M, int N, int K);
cudaError_t launch_gemm(const GemmArgs &a, cudaStream_t stream);

// The same for a few rows of K-major operands, the contraction a multiple of 8.
inline bool small_gemm_ok(int M, int K) { return M <= 16 && K % 8 == 0; }
cudaError_t launch_small_gemm(const GemmArgs &a, cudaStream_t stream);

// Rows copied to such boundaries: dst's rows are ld elements apart, a multiple of 8.
struct CopyArgs {
    const void *src;
    void *dst;
    long long rows, lds, ldd;
    int width;
    unsigned *dbg;
};
cudaError_t launch_copy_rows(const CopyArgs &a, const CopyArgs *b, cudaStream_t stream);  // b: or null

// dpre = dy act'(pre) (dpre null: not wanted) and its column sums (dbias null: not wanted).
struct DActArgs {
    const void *dy, *pre;
    void *dpre, *dbias;
    float *partial;  // [dact_partials(M, N)][N]
    size_t partial_floats;
    long long lddy, ldp, ldd;
    int M, N, act;
    bool fp16;
    unsigned *dbg;
};
int dact_partials(int M, int N);
cudaError_t launch_dact(const DActArgs &a, cudaStream_t stream);

}  // namespace kda
