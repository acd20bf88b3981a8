// Internal launch interface of the recurrence, single-token and layer-norm operators.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace kda {

constexpr int kSMs = 152;

struct ChunkFwdArgs {
    const void *q, *k, *v;  // 16-bit, [rows, H, 128] and [rows, HV, 128]
    const float *gate, *beta;
    void *o;
    const float *initial_state;  // [num_seqs, HV, 128 dk, 128 dv] or null
    float *final_state;          // the same, or null
    char *ckpt, *e, *tiles;      // the backward's buffers, all or none
    float *scales;               // with them in BF16 training (kda_fast.cuh)
    int T, H, HV, num_seqs;      // T = tokens of a sequence, or of the packed row
    const int *cu_seqlens;       // [num_seqs + 1] or null
    float scale;
    bool fp16;
    bool fast;                   // BF16 training (kda_fast.cuh)
    // For the debug build's checks: rows of o (tokens * HV), slots of value heads that are saved,
    // elements of a state's tensor.
    size_t rows_o, units, states;
    unsigned *dbg;
};

cudaError_t launch_chunk_fwd(const ChunkFwdArgs &a, cudaStream_t stream);

struct ChunkBwdArgs {
    const void *q, *k, *dout;  // 16-bit
    const float *gate, *beta;
    void *dq, *dk, *dv, *dgate, *dbeta;  // 16-bit; dq, dk [rows, H, 128]
    const float *d_final_state;          // [num_seqs, HV, 128 dk, 128 dv] or null
    float *d_initial_state;              // the same, or null
    const char *ckpt, *e, *tiles;        // what the forward saved
    const float *scales;
    char *dckpt, *y;                     // workspace: state gradients at slot ends, Y
    float *dscales;
    bool fast;                           // BF16 training (kda_fast.cuh)
    float *dq_hv, *dk_hv;                // workspace [rows, HV, 128], only when HV > H
    bool gates32;                        // dgate and dbeta are FP32
    int B, T, H, HV, num_seqs, slots;
    const int *cu_seqlens;
    float scale;
    bool fp16;
    size_t rows_o, units, states;  // as above
    unsigned *dbg;
};

cudaError_t launch_chunk_bwd(const ChunkBwdArgs &a, cudaStream_t stream);

// Outputs [T, row bytes] of a packed call, whose tokens in no sequence get zeros.
struct ZeroArgs {
    void *out[5];
    size_t row[5];
    int count, T, num_seqs;
    const int *cu_seqlens;
    unsigned *dbg;
};

cudaError_t launch_zero_rest(const ZeroArgs &a, cudaStream_t stream);

struct StepArgs {
    const void *q, *k, *v;  // 16-bit, [N, H, 128] and [N, HV, 128]
    const float *gate, *beta;
    float *state;           // [num_states, HV, 128 dk, 128 dv]
    void *o;
    int N, H, HV;
    const int *state_indices;  // [N] or null (request n has state n)
    long long num_states;
    float scale;
    bool fp16;
    unsigned *dbg;
};

cudaError_t launch_step(const StepArgs &a, cudaStream_t stream);

// Element types of the layer norm's tensors.
enum { NORM_BF16 = 0, NORM_FP16 = 1, NORM_FP32 = 2 };

struct NormArgs {
    const void *x, *weight, *bias;  // weight, bias: null = ones, zeros
    void *y;
    float *mean, *rstd;             // [rows]; forward: null = not wanted
    // backward
    const void *dy;
    void *dx;
    float *dweight, *dbias;         // [width], both or none
    float *partial;                 // [partials = norm_bwd_ctas(rows, width)][2][width]
    int partials;
    long long rows;
    int width, dtype, wdtype;
    long long x_stride, y_stride, dy_stride, dx_stride;  // elements between rows
    float eps;
    unsigned *dbg;
};

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t stream);
int norm_bwd_ctas(long long rows, int width);  // rows of `partial`

}  // namespace kda
