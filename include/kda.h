/*
 * libkda -- intra-chunk backward of chunked KDA (Kimi Delta Attention, the gated
 * delta rule with a per-channel gate) on sm_103a.
 *
 * What it computes (bwd_intra page: the module docstring of kernel_fun/kda/_kernels/
 * bwd_intra.py, its diagonal and epilogue loops, and the host wrapper's tensor
 * contract).  Tokens are cut into chunks of KDA_BT = 64; a "unit" is one
 * (batch b, head h, chunk c).  Inside a unit, with rows r, s in [0, 64), channels
 * d in [0, 128) and E[r,s,d] = 2^(g[r,d] - g[s,d]):
 *
 *   Aqk[r,s] = sum_d q[r,d] k[s,d] E[r,s,d]             (s <= r)
 *   Akk[r,s] = beta[r] * sum_d k[r,d] k[s,d] E[r,s,d]   (s <  r)
 *
 * Given the upstream gradients dAqk and dAkk, the library returns the gradients
 * of L = sum dAqk*Aqk + sum dAkk*Akk with respect to q, k, beta and g:
 *
 *   dq[r]   = sum_{s<=r} dAqk[r,s] k[s] E[r,s]
 *   dk[t]   = beta[t] sum_{s<t} dAkk[t,s] k[s] E[t,s]
 *             + sum_{r>=t} (dAqk[r,t] q[r] + [r>t] dAkk[r,t] beta[r] k[r]) E[r,t]
 *   db[r]   = sum_{s<r} dAkk[r,s] sum_d k[r,d] k[s,d] E[r,s,d]
 *   dg[t]   = ln2 * ( q[t] (dq[t]) + (beta[t] acck[t] - dkt[t]) k[t] )
 *             where acck[t] = sum_{s<t} dAkk[t,s] k[s] E[t,s] and dkt[t] is the
 *             second line of dk[t]  (all products per channel d)
 *
 * dg is the gradient with respect to g exactly as passed (a log2 cumulative gate):
 * it is the bwd_intra page's epilogue value times ln2.  A caller whose gate lives
 * in natural-log units (g_nat = g * ln2) gets dL/dg_nat as dg / ln2.
 *
 * Supported shapes: K = 128 (head dimension), chunk 64; fixed-length sequences with
 * T a multiple of 64, or (kda_intra_bwd_ex only) variable-length sequences packed
 * along T and described by cu_seqlens.  g must be the inclusive chunk-local
 * cumulative sum of per-step log2 gates that are <= 0 (non-increasing inside each
 * chunk): every exponent the kernels evaluate is then <= 0.
 *
 * Memory: every pointer is caller-owned DEVICE memory (except the *_host entry
 * point), contiguous row-major, 16-byte aligned, and must not overlap another
 * argument:
 *   q, k        [B, T, H, 128]  bf16 or fp16 (qk_dtype)
 *   g           [B, T, H, 128]  fp32
 *   beta        [B, T, H]       fp32
 *   dAqk, dAkk  [B, T, H, 64]   fp32; row = token, column = source index inside the
 *                               token's chunk.  Entries outside the support (dAqk
 *                               above the diagonal, dAkk on or above it) are ignored.
 *   dq, dk, dg  [B, T, H, 128]  fp32 outputs, fully overwritten
 *   db          [B, T, H]       fp32 output, fully overwritten
 *
 * Calls are asynchronous on `stream` (0 = the legacy default stream): no host
 * synchronisation and no device allocation happens inside.  Inputs are not modified.
 * Argument errors are reported before anything is launched; no call aborts the
 * process.
 *
 * Stalled pipelines: every wait of a kernel on its own copies or tensor-core work is
 * bounded (about 4M polls).  A wait that gives up does not hang or trap: the kernel
 * writes NaN into the outputs of the unit it was working on and carries on (the matrix
 * product: NaN into all that this block of threads had still to write).  The call
 * has already returned KDA_OK when this happens (the status only covers the arguments
 * and the launch), so in the normal build a stalled pipeline is seen only as NaN
 * outputs, which NaN or Inf inputs can also produce.  The bounds-checked debug build
 * (kda_debug_set_flags below) also sets KDA_DBG_WAIT in its flag word, which tells the
 * two apart.  No valid input makes a wait give up on a healthy GPU.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ABI versions (kda_abi_version() returns the loaded library's):
 *   13 kda_debug_set_give_up, KDA_DBG_SHORT
 *   12 kda_conv_fwd, kda_conv_bwd, kda_conv_step, kda_scan_fwd, kda_scan_bwd, kda_scan_step,
 *      kda_linear_fwd, kda_linear_bwd and their option structs and size queries
 *   11 kda_chunk_bwd's zero_rest also takes KDA_GATE_GRADS_FP32, kda_chunk_fwd's saved either
 *      of its sizes in BF16 calls without a state
 *   10 kda_chunk_fwd, kda_chunk_bwd, kda_step, kda_layer_norm_fwd, kda_layer_norm_bwd
 *      and their option structs and size queries
 *   9  kda_intra_bwd_opts_t gains split_tf32 (appended; the struct grew)
 *   8  kda_intra_bwd_host_static, KDA_HOST_STATIC_MAX_BYTES, KDA_ERR_TOO_LARGE
 *   7  kda_debug_checks, kda_debug_set_flags (the bounds-checked debug build)
 *   6  kda_intra_bwd_opts_t gains factor_diag (appended; the struct grew)
 *   5  kda_intra_fwd_ex and kda_intra_fwd_opts_t
 *   4  kda_intra_fwd
 *   3  variable-length fields of kda_intra_bwd_opts_t (cu_seqlens .. num_chunks)
 *   2  kda_intra_bwd_ex and kda_intra_bwd_opts_t
 *   1  kda_intra_bwd, kda_intra_bwd_fp32, the host entry point, status helpers
 * Option structs only grow at their end, and the library reads sizeof(its own struct)
 * from the pointer it is given.  A caller compiled against an older header would have
 * the library read past the end of its struct, so a caller that passes an option struct
 * must check at start-up that kda_abi_version() equals the KDA_ABI_VERSION it was
 * compiled with (the Python binding refuses to load any other version).
 */
#define KDA_ABI_VERSION 13
#define KDA_BT 64  /* chunk length */
#define KDA_BC 16  /* sub-block length inside a chunk */
#define KDA_K 128  /* head dimension */
#define KDA_MAX_H 65536 /* largest supported head count */

/* Same type as cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st *kda_stream_t;

typedef enum {
    KDA_OK = 0,
    KDA_ERR_NULL = 1,               /* a required pointer is NULL */
    KDA_ERR_SHAPE = 2,              /* B,T,H <= 0, H > KDA_MAX_H, T % 64 != 0, too large;
                                       varlen: B != 1, num_seqs <= 0, num_chunks < 0 */
    KDA_ERR_DTYPE = 3,              /* qk_dtype not KDA_BF16 / KDA_FP16 */
    KDA_ERR_ALIGN = 4,              /* a pointer is not 16-byte aligned */
    KDA_ERR_CUDA = 5,               /* a CUDA runtime call or the launch failed */
    KDA_ERR_UNSUPPORTED_DEVICE = 6, /* current device is not compute capability 10.3 */
    KDA_ERR_OVERLAP = 7,            /* two argument buffers overlap */
    KDA_ERR_WORKSPACE = 8,          /* workspace missing or too small (*_host only) */
    KDA_ERR_OPTION = 9,             /* unsupported option combination (*_ex), or debug
                                       reporting asked of a build without checks */
    KDA_ERR_TOO_LARGE = 10          /* the call needs more scratch than the library's
                                       fixed KDA_HOST_STATIC_MAX_BYTES
                                       (kda_intra_bwd_host_static only) */
} kda_status_t;

typedef enum { KDA_BF16 = 0, KDA_FP16 = 1 } kda_dtype_t;

/*
 * The intra-chunk backward, fast path: 16x16 diagonal sub-blocks on the FP32 pipes
 * with one exp2 per (r, s, d); the cross-sub-block sums factorized through each
 * sub-block's boundary gate (every exp2 argument <= 0) and contracted on the
 * tensor cores in TF32 with FP32 accumulation.  Accuracy: max|err| / max|ref|
 * <= 2e-3 per output tensor against the fp64 definition.
 */
kda_status_t kda_intra_bwd(const void *q, const void *k, const float *g,
                           const float *beta, const float *dAqk, const float *dAkk,
                           float *dq, float *dk, float *db, float *dg,
                           int B, int T, int H, kda_dtype_t qk_dtype,
                           kda_stream_t stream);

/*
 * Same contract, every product and sum in FP32 (the cross-sub-block sums on the
 * FP32 pipes through the same boundary factorization).  Slower; accuracy
 * max|err| / max|ref| <= 1e-4 per output tensor.
 */
kda_status_t kda_intra_bwd_fp32(const void *q, const void *k, const float *g,
                                const float *beta, const float *dAqk, const float *dAkk,
                                float *dq, float *dk, float *db, float *dg,
                                int B, int T, int H, kda_dtype_t qk_dtype,
                                kda_stream_t stream);

/*
 * End-to-end convenience for callers holding HOST buffers: copies the six inputs
 * into `workspace` (device memory of at least kda_intra_bwd_host_workspace_bytes()
 * bytes, caller-owned, 256-byte aligned), runs kda_intra_bwd, and copies the four
 * outputs back into the host buffers.  The work is pipelined over pieces of about
 * 96 MB of input (whole 64-token chunks; beta goes up whole before the first piece
 * and db comes down whole after the last): uploads run on one internal stream,
 * downloads on another and the kernels on `stream`, so both copy directions and the
 * compute overlap; events order it all after earlier work on `stream`, and `stream`
 * waits for the last copy of each direction (also when a call fails midway).  The two
 * internal streams and their events are made by the first call on each device and
 * kept until the process exits; calls from several threads queue their work one call
 * after another on them.  Copies are truly asynchronous only when the host buffers
 * are page-locked.  The call returns once everything is queued: synchronise
 * `stream` before reading the outputs or reusing the inputs.  Host pointers need no
 * particular alignment.
 */
size_t kda_intra_bwd_host_workspace_bytes(int B, int T, int H, kda_dtype_t qk_dtype);

kda_status_t kda_intra_bwd_host(const void *q, const void *k, const float *g,
                                const float *beta, const float *dAqk, const float *dAkk,
                                float *dq, float *dk, float *db, float *dg,
                                int B, int T, int H, kda_dtype_t qk_dtype,
                                void *workspace, size_t workspace_bytes,
                                kda_stream_t stream);

/*
 * kda_intra_bwd_host without a workspace argument, for callers that hold only host
 * buffers and may not allocate device memory: a plugin or FFI caller inside a host
 * application whose device memory is owned by another allocator (a framework's
 * caching pool that has reserved it, a fixed per-process budget), or code on a
 * latency-critical path where cudaMalloc's implicit device synchronisation is not
 * acceptable.  The paper has no counterpart for this entry point; it is a deployment
 * convenience around the same kernel.
 *
 * The device staging buffers live in one array of this library, KDA_HOST_STATIC_MAX_BYTES
 * (32 MiB) of global memory that every GPU on which the library's device code is loaded
 * holds until the process exits.  A call whose staging need,
 * kda_intra_bwd_host_workspace_bytes(B, T, H, qk_dtype), exceeds it returns
 * KDA_ERR_TOO_LARGE before anything is queued.  The need is 3080 bytes per token-head
 * row, so up to B*T*H = 10,880 rows fit (for instance B = 2, T = 1024, H = 4); larger
 * problems take kda_intra_bwd_host with a caller-owned workspace.  The call allocates
 * nothing (no cudaMalloc, no cudaFree, no stream, no event): it queues the six uploads,
 * the kernel and the four downloads, in that order, on `stream` and returns.
 * Synchronise `stream` before reading the outputs or reusing the inputs.
 *
 * The first call on each device looks up the array's device address (with that device
 * current); make that first call before any stream capture on that device.  Every call,
 * on every stream and thread, shares the one array: calls whose work overlaps on the GPU
 * race on it, so order them on one stream (or synchronise between them).  The array keeps
 * the last call's contents; nothing in it needs to start at zero, since each call
 * overwrites every byte it reads.  Same arguments, status codes and accuracy as
 * kda_intra_bwd_host otherwise.
 */
#define KDA_HOST_STATIC_MAX_BYTES 33554432u /* 32 MiB */

kda_status_t kda_intra_bwd_host_static(const void *q, const void *k, const float *g,
                                       const float *beta, const float *dAqk,
                                       const float *dAkk, float *dq, float *dk,
                                       float *db, float *dg, int B, int T, int H,
                                       kda_dtype_t qk_dtype, kda_stream_t stream);

/*
 * Options of kda_intra_bwd_ex.  Zero-initialise, then set what you need; a zeroed
 * struct (or a NULL pointer) gives exactly kda_intra_bwd.  These follow the bwd_intra
 * page's host wrapper and kernel options (its incoming-gradient tensors, fold_dg,
 * emit_bf16 and gva group size).
 *
 *   HV             heads of g, beta, dAqk, dAkk and of every output and *_in tensor;
 *                  q and k keep H heads and value head hv reads q/k head hv / (HV / H)
 *                  (grouped value attention).  0 means HV = H.  Must be a multiple of H.
 *   dq_in, dk_in,  optional [B,T,HV,128] fp32 gradients added in-kernel to dq, dk, dg
 *   dg_in          (NULL = none).  May be the same pointer as the matching output
 *                  (in-place accumulation); any other overlap is rejected.  When dq_in,
 *                  dk_in and (without fold_dg) dg_in are all their outputs, the kernel
 *                  reads none of them: its stores add to them in L2 (red.global.add, one
 *                  rounding as otherwise, but subnormal sums flush to zero), the fastest
 *                  way to accumulate.
 *   db_in          optional [B,T,HV] fp32 added to db; may equal db.
 *   fold_dg        1: dg comes back as its inclusive reverse cumsum inside each
 *                  64-token chunk, out[t] = sum_{t' >= t in t's chunk} dg[t'] (the
 *                  per-step gate's gradient; dg_in is added before the fold).
 *   dqdk_io_dtype  1: dq and dk are written in qk_dtype (round to nearest) instead of
 *                  fp32 -- bitwise the cast of the fp32 result.  Not allowed with HV > H
 *                  (the grouped-head reduction that follows must see fp32 values).
 *   cu_seqlens     variable-length sequences (the host wrapper's cu_seqlens /
 *   chunk_indices  chunk_indices pair).  B must be 1 and T is the packed token count
 *   num_seqs       (any T >= 1).  cu_seqlens: device int32 [num_seqs + 1], sequence n
 *   num_chunks     is tokens [cu_seqlens[n], cu_seqlens[n+1]), 0 = cu_seqlens[0] <=
 *                  ... <= cu_seqlens[num_seqs] <= T.  chunk_indices: device int32
 *                  [num_chunks][2], entry c = (n, j) names chunk j of sequence n, i.e.
 *                  tokens cu_seqlens[n] + 64j ... min(+64, cu_seqlens[n+1]) - 1; chunks
 *                  restart at every sequence start, and a sequence's last chunk may be
 *                  short.  Each unit is then (chunk entry, head); all per-chunk
 *                  definitions above apply to the chunk's valid rows only (g is the
 *                  cumsum restarted at each chunk start, dA rows are indexed from the
 *                  chunk start, fold_dg folds over the valid rows).  Both pointers are
 *                  NULL for fixed-length calls (chunk_indices may also be NULL when
 *                  num_chunks == 0: nothing is launched); the rows of tokens that no entry names
 *                  are left untouched.  The values are read on the device only: an
 *                  entry that names no chunk of cu_seqlens (n out of range, j past the
 *                  sequence's end, a sequence past T) is skipped, so no input value can
 *                  make the kernel access memory outside the argument buffers.
 *   factor_diag    0: every pair of a 16x16 diagonal block takes its own exp2, one per
 *                  (r, s, d), as in kda_intra_bwd.  1: the lower-left 8x8 quadrant of
 *                  each diagonal block (rows 8..15 against sources 0..7 of the block) is
 *                  factorized through the block's row 8, 2^(g_r - g_s) =
 *                  2^(g_r - g_8) * 2^(g_8 - g_s); both exponents are <= 0 (g is
 *                  non-increasing inside a chunk), so nothing can overflow, and the
 *                  quadrant costs four FMAs per (r, s, d) instead of an exp2 and seven
 *                  FP32 operations (about 4% less kernel time).  The result differs
 *                  from the exact form by rounding only; same accuracy contract.
 *   split_tf32     1: the cross-sub-block sums in split TF32 for FP32-level accuracy:
 *                  every tensor-core operand x is cut into hi = tf32(x) and lo = x - hi
 *                  and each product is taken as A_hi B_hi + A_hi B_lo + A_lo B_hi on the
 *                  tensor cores with FP32 accumulation (the dropped A_lo B_lo is about
 *                  2^-22 of the product); the diagonal blocks stay on the FP32 pipes.
 *                  Accuracy max|err| / max|ref| <= 1e-4 per output tensor, as
 *                  kda_intra_bwd_fp32, at about half its time.  Fixed-length sequences
 *                  only, and no other option but HV; anything else is KDA_ERR_OPTION.
 *
 * Runs on the tensor-core path (the same accuracy contract as kda_intra_bwd, except
 * with split_tf32).
 */
typedef struct {
    int HV;
    const float *dq_in;
    const float *dk_in;
    const float *dg_in;
    const float *db_in;
    int fold_dg;
    int dqdk_io_dtype;
    const int *cu_seqlens;
    const int *chunk_indices;
    int num_seqs;
    int num_chunks;
    int factor_diag;
    int split_tf32;
} kda_intra_bwd_opts_t;

kda_status_t kda_intra_bwd_ex(const void *q, const void *k, const float *g,
                              const float *beta, const float *dAqk, const float *dAkk,
                              void *dq, void *dk, float *db, float *dg,
                              int B, int T, int H, kda_dtype_t qk_dtype,
                              const kda_intra_bwd_opts_t *opts, kda_stream_t stream);

/*
 * The intra-chunk forward: the two score matrices whose gradients kda_intra_bwd
 * takes, for every unit (b, h, 64-token chunk) and rows r, s of the chunk,
 *
 *   Aqk[r,s] = sum_d q[r,d] k[s,d] E[r,s,d]             (s <= r, else 0)
 *   Akk[r,s] = beta[r] * sum_d k[r,d] k[s,d] E[r,s,d]   (s <  r, else 0)
 *
 * (same definitions as above).  q, k, g, beta as for kda_intra_bwd; Aqk and Akk are
 * [B, T, H, 64] fp32 device outputs, fully overwritten (zeros outside the support),
 * 16-byte aligned, not overlapping anything else.  Cross-sub-block entries come from
 * TF32 tensor-core products through the boundary factorization (every exp2 argument
 * <= 0), the diagonal 16x16 blocks from FP32 with one exp2 per (r, s, d).
 * Accuracy: max|err| / max|ref| <= 2e-3 per output tensor.  Same shape rules, status
 * codes and asynchrony as kda_intra_bwd.
 */
kda_status_t kda_intra_fwd(const void *q, const void *k, const float *g,
                           const float *beta, float *Aqk, float *Akk,
                           int B, int T, int H, kda_dtype_t qk_dtype,
                           kda_stream_t stream);

/*
 * Options of kda_intra_fwd_ex (zero-initialise; a zeroed struct or NULL gives exactly
 * kda_intra_fwd), with the meanings of kda_intra_bwd_opts_t:
 *   HV             heads of g, beta, Aqk and Akk; q and k keep H heads, and value head
 *                  hv reads q/k head hv / (HV / H).  0 means HV = H.
 *   cu_seqlens,    variable-length sequences packed along T (B == 1, any T >= 1):
 *   chunk_indices, the same tables and the same checks as for the backward.  Rows of
 *   num_seqs,      a chunk past its sequence's end take no part in any valid entry and
 *   num_chunks     are not written; tokens no entry names are left untouched.
 */
typedef struct {
    int HV;
    const int *cu_seqlens;
    const int *chunk_indices;
    int num_seqs;
    int num_chunks;
} kda_intra_fwd_opts_t;

kda_status_t kda_intra_fwd_ex(const void *q, const void *k, const float *g,
                              const float *beta, float *Aqk, float *Akk,
                              int B, int T, int H, kda_dtype_t qk_dtype,
                              const kda_intra_fwd_opts_t *opts, kda_stream_t stream);

/*
 * The gated delta-rule recurrence over whole sequences.  Per value head the state S is
 * [128 dk, 128 dv]; a token first decays it per channel, then corrects it towards its value:
 *
 *   S~_t = diag(2^gate_t) S_{t-1},   e_t = v_t - S~_t^T k_t,
 *   S_t  = S~_t + beta_t k_t e_t^T,  o_t = scale S_t^T q_t
 *
 * (the intra-chunk step above is what this recurrence is made of inside a chunk).  All
 * pointers are device memory, contiguous row-major, 16-byte aligned (beta: 4):
 *   q, k        [B, T, H, 128]   bf16 or fp16 (dtype)
 *   v, o        [B, T, HV, 128]  dtype; o fully overwritten
 *   gate        [B, T, HV, 128]  fp32 per-step log2 decay, <= 0 (NOT cumulative; the
 *                                kda_intra_* calls take its chunk-local cumsum).  Values below
 *                                -160, the type's lowest and -infinity among them, clear the
 *                                channel.
 *   beta        [B, T, HV]       fp32
 * HV is a multiple of H; value head hv reads q/k head hv / (HV / H).  Any T >= 0.
 *
 * Accuracy (2-norm of the error over 2-norm of the result, of some dozen tokens; of a few whose
 * q.k or S^T q cancels, that share of |q| |k| |v| and |S| |q|): states, sums and the solve are
 * FP32.  Calls that take or return a state, and FP16 ones, take every product of FP32 values
 * in three BF16 tensor-core products: o within a rounding to dtype plus 1e-5, the final state
 * within 1e-5 (up to twice that when it holds a few tokens only).  BF16 calls without a state
 * (training) take one FP16 product with operands of 11 bits, each with a power of two of its
 * own: o within a rounding to BF16 plus 1e-3, for values between 2^-80 and 2^100.  q and k have
 * one power each a step of 16 tokens: of a token below 2^-6 of the step's largest bits are lost.
 * A caller who wants the former there passes `saved` of a call with a state (or takes the final
 * state): the size chooses.
 *
 * Options (zero-initialise; NULL = none):
 *   HV             0 means HV = H
 *   scale          0 means 128^-0.5
 *   initial_state  [sequences, HV, 128 dk, 128 dv] fp32, NULL = zeros
 *   final_state    the same shape, written (a sequence of no tokens: a copy of its initial
 *                  state); must not overlap initial_state
 *   saved          what kda_chunk_bwd needs, exactly kda_chunk_saved_bytes() bytes, 256-byte
 *   saved_bytes    aligned; NULL when no backward follows.  0.9 KB a token and value head in
 *                  BF16 without a state, 1.7 KB otherwise (with_state = 1, which a BF16 call
 *                  without a state may have too).
 *   cu_seqlens     variable-length sequences packed along T (B == 1): device int32
 *   num_seqs       [num_seqs + 1], sequence n is tokens [cu_seqlens[n], cu_seqlens[n+1]).
 *                  Values are read on the device only and clamped to [0, T]; tokens in no
 *                  sequence are left untouched, or with
 *   zero_rest      get zeros.
 */
typedef struct {
    int HV;
    float scale;
    const float *initial_state;
    float *final_state;
    void *saved;
    size_t saved_bytes;
    const int *cu_seqlens;
    int num_seqs;
    int zero_rest;
} kda_chunk_fwd_opts_t;

/* Bytes of `saved` (num_seqs: 0 for fixed-length calls; with_state: whether the call has an
 * initial_state or a final_state); 0 for sizes that no call accepts. */
size_t kda_chunk_saved_bytes(int B, int T, int HV, int num_seqs, kda_dtype_t dtype,
                             int with_state);

kda_status_t kda_chunk_fwd(const void *q, const void *k, const void *v, const float *gate,
                           const float *beta, void *o, int B, int T, int H, kda_dtype_t dtype,
                           const kda_chunk_fwd_opts_t *opts, kda_stream_t stream);

/*
 * Gradients of kda_chunk_fwd from dout [B, T, HV, 128] (dtype) and what it saved: dq, dk
 * [B, T, H, 128] (summed over the value heads of a q/k head), dv, dgate [B, T, HV, 128] and
 * dbeta [B, T, HV], all in dtype, rounded once from FP32 sums; all 16-byte aligned but beta (4)
 * and dbeta (2).  q, k, gate, beta, scale, HV and cu_seqlens as given to the forward (zero_rest
 * as there, for all five).  No atomics: the same inputs give the same bits.
 *   zero_rest        1 and, or alone, KDA_GATE_GRADS_FP32: dgate and dbeta are fp32 (dbeta then
 *                    4-byte aligned), not rounded to dtype
 *   d_final_state    gradient of the final state, [sequences, HV, 128, 128] fp32, NULL = zeros
 *   d_initial_state  gradient of the initial state, the same shape, written; NULL = not wanted
 *   saved            the forward's, read only (a backward may run again from it); saved_bytes
 *                    is the forward's too, and tells how it was written
 *   workspace        kda_chunk_bwd_workspace_bytes() bytes, 256-byte aligned
 * Accuracy: within a rounding to dtype plus 1e-4, the initial state's gradient within 1e-5;
 * after a BF16 forward that took the 11-bit operands a rounding plus 1e-3 (and 1e-3).  dgate and
 * dbeta are sums that may cancel: what they are within is then that share of their terms (of
 * |q dq| + |k dk|, and of |dv / beta| |v - S~^T k|).
 */
#define KDA_GATE_GRADS_FP32 2

typedef struct {
    int HV;
    float scale;
    const float *d_final_state;
    float *d_initial_state;
    const int *cu_seqlens;
    int num_seqs;
    int zero_rest;
    const void *saved;
    size_t saved_bytes;
    void *workspace;
    size_t workspace_bytes;
} kda_chunk_bwd_opts_t;

size_t kda_chunk_bwd_workspace_bytes(int B, int T, int H, int HV, int num_seqs,
                                     kda_dtype_t dtype, size_t saved_bytes);

kda_status_t kda_chunk_bwd(const void *q, const void *k, const float *gate, const float *beta,
                           const void *dout, void *dq, void *dk, void *dv, void *dgate,
                           void *dbeta, int B, int T, int H, kda_dtype_t dtype,
                           const kda_chunk_bwd_opts_t *opts, kda_stream_t stream);

/*
 * One token of the recurrence for each of N requests (serving): o [N, HV, 128] from q, k
 * [N, H, 128], v [N, HV, 128], gate [N, HV, 128], beta [N, HV]; each request's state in
 * `state` [num_states, HV, 128 dk, 128 dv] fp32 is updated in place.  state_indices (device
 * int32 [N], NULL = request n has state n) names the states; no two requests may name the
 * same one, and an index outside [0, num_states) marks a row without a request (a padded
 * batch): its o is zero and no state is touched.  scale 0 means 128^-0.5.  FP32 throughout.
 */
typedef struct {
    int HV;
    float scale;
    const int *state_indices;
    int num_states; /* 0 means N */
} kda_step_opts_t;

kda_status_t kda_step(const void *q, const void *k, const void *v, const float *gate,
                      const float *beta, float *state, void *o, int N, int H, kda_dtype_t dtype,
                      const kda_step_opts_t *opts, kda_stream_t stream);

/*
 * Layer norm over the last dimension of x [rows, width] (any width >= 1):
 *   y = (x - mean) rstd weight + bias,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 * x, y, dy and dx have one type (KDA_BF16, KDA_FP16 or KDA_FP32) and a row stride each, in
 * elements (0 = width); weight and bias have `wdtype`, which is the same type or KDA_FP32, and
 * may be NULL (ones, zeros).  mean and rstd [rows] fp32 are what the backward needs (NULL =
 * not wanted).  y and dx must not overlap the inputs; column slices of one buffer may lie side by
 * side.  Statistics, sums and gradients of weight and bias are FP32.  Pointers need
 * their element's alignment; rows on 16-byte boundaries are read and written 16 bytes at a
 * time, others element by element.
 *
 * Backward: dx, and dweight, dbias [width] fp32 (both or neither), summed over the rows in a
 * fixed order.  `workspace` holds kda_layer_norm_bwd_workspace_bytes() bytes of partial sums
 * (16-byte aligned; not needed without dweight).
 */
#define KDA_FP32 2 /* layer norm, convolution and scan */

kda_status_t kda_layer_norm_fwd(const void *x, const void *weight, const void *bias, void *y,
                                float *mean, float *rstd, long long rows, int width, float eps,
                                int dtype, int wdtype, long long x_stride, long long y_stride,
                                kda_stream_t stream);

size_t kda_layer_norm_bwd_workspace_bytes(long long rows, int width);

kda_status_t kda_layer_norm_bwd(const void *dy, const void *x, const void *weight,
                                const float *mean, const float *rstd, void *dx, float *dweight,
                                float *dbias, long long rows, int width, int dtype, int wdtype,
                                long long dy_stride, long long x_stride, long long dx_stride,
                                void *workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * Short causal convolution of each channel (the one in front of q, k and v, or of the scan below):
 *   pre[t, d] = bias[d] + sum_j weight[d, j] x[t - W + 1 + j, d],  y = act(pre)
 * over the tokens of a sequence, x, y [B, T, D] with a row stride each, in elements (0 = D), W 2 to
 * 4, D up to 2^28.  x, y, dy, dx and the states have one type (KDA_BF16, KDA_FP16 or KDA_FP32); weight [D, W] and
 * bias [D] (NULL = 0) have `wdtype`, which is the same type or KDA_FP32.  The inputs in front of a
 * sequence come from initial_state [sequences, W - 1, D], oldest first (NULL = zeros); final_state
 * gets the last W - 1 of state and sequence (a sequence of no tokens: a copy).  Sums are FP32.
 * cu_seqlens, num_seqs and zero_rest as in kda_chunk_fwd (zero_rest: rows of outputs D apart).
 * Pointers need their element's alignment; channels on 16-byte boundaries are read 16 bytes at a
 * time.
 *
 * Backward: dx, and dweight [D, W], dbias [D] fp32 (both or neither), summed over the tokens in a
 * fixed order; d_final_state (NULL = zeros) and d_initial_state (written, NULL = not wanted)
 * are like the states.  `workspace` holds kda_conv_bwd_workspace_bytes() bytes,
 * 16-byte aligned (not needed without dweight).
 *
 * kda_conv_step: one token for each of N <= 65535 requests, x, y [N, D], `state` [num_states, W - 1,
 * D] updated in place; state_indices as in kda_step.
 */
#define KDA_ACT_NONE 0
#define KDA_ACT_SILU 1
#define KDA_ACT_GELU 2 /* x Phi(x), of the matrix product only */
#define KDA_ACT_RELU 3 /* of the matrix product only */

typedef struct {
    const void *initial_state;
    void *final_state;
    const int *cu_seqlens;
    int num_seqs;
    int zero_rest;
    long long x_stride, y_stride;
} kda_conv_fwd_opts_t;

kda_status_t kda_conv_fwd(const void *x, const void *weight, const void *bias, void *y, int B, int T,
                          int D, int W, int dtype, int wdtype, int activation,
                          const kda_conv_fwd_opts_t *opts, kda_stream_t stream);

typedef struct {
    const void *initial_state, *d_final_state;
    void *d_initial_state;
    const int *cu_seqlens;
    int num_seqs;
    int zero_rest;
    long long dy_stride, x_stride, dx_stride;
    void *workspace;
    size_t workspace_bytes;
} kda_conv_bwd_opts_t;

size_t kda_conv_bwd_workspace_bytes(int B, int T, int D, int W, int num_seqs);

kda_status_t kda_conv_bwd(const void *dy, const void *x, const void *weight, const void *bias, void *dx,
                          float *dweight, float *dbias, int B, int T, int D, int W, int dtype,
                          int wdtype, int activation, const kda_conv_bwd_opts_t *opts,
                          kda_stream_t stream);

typedef struct {
    const int *state_indices;
    int num_states; /* 0 means N */
    long long x_stride, y_stride;
} kda_conv_step_opts_t;

kda_status_t kda_conv_step(const void *x, const void *weight, const void *bias, void *state, void *y,
                           int N, int D, int W, int dtype, int wdtype, int activation,
                           const kda_conv_step_opts_t *opts, kda_stream_t stream);

/*
 * Selective state-space scan.  Per channel d of D a state h of N <= 64 numbers (D and G N up to 2^28):
 *   s_t = softplus(delta_t + delta_bias)              (plain_delta: without the softplus)
 *   h_t[n] = exp(s_t A[d, n]) h_{t-1}[n] + s_t u_t B_t[n],
 *   y_t = (sum_n C_t[n] h_t[n] + skip[d] u_t) silu(z_t)
 * u, delta, z, y [B, T, D], Bm, Cm [B, T, G, N] (channel d reads group d / (D / G)), all of one type
 * (KDA_BF16, KDA_FP16 or KDA_FP32) with a row stride each, in elements (0 = D, G N); A [D, N], skip,
 * delta_bias [D] fp32.  skip, z, delta_bias: NULL = none.  A is finite, <= 0 for states that fade.
 * Pointers need their element's alignment (rows on boundaries of four elements are read
 * four channels at a time), saved and workspace 256 bytes.  States, sums and exponentials are FP32: a token's
 * decay is off by 3e-9 of the state on the mean (1.4e-8 of states that last 250 tokens or less) and by 3e-8 at
 * random (by the same number at every token where delta never changes, 8e-8 at most), which a state adds up
 * over the tokens that it lasts.
 *   initial_state, final_state   [sequences, D, N] fp32 as in kda_chunk_fwd
 *   saved, saved_bytes           what kda_scan_bwd needs: kda_scan_saved_bytes(), N / 2 bytes a token and
 *                                channel for states (N rounded up to 8, 16, 32 or 64, each sequence's
 *                                tokens to 16, of packed ones 16 more) and 4 for what the gate
 *                                multiplies, which are there, unused, without z too; NULL when no
 *                                backward follows
 *   cu_seqlens, num_seqs,        as in kda_chunk_fwd (zero_rest: rows of y D apart)
 *   zero_rest
 *   workspace                    kda_scan_fwd_workspace_bytes() bytes (0 where the card is full of
 *                                channels)
 *
 * kda_scan_bwd: du, ddelta, dz [B, T, D], dB, dC [B, T, G, N] of the type, contiguous, rounded once;
 * dA [D, N], dskip, ddelta_bias [D] fp32.  dz, dskip and ddelta_bias come with z, skip and
 * delta_bias.  No atomics: the same inputs give the same bits.  zero_rest: for all five outputs
 * with rows of tokens.
 *
 * kda_scan_step: one token for each of `requests` <= 65535: u, delta, z, y [requests, D], Bm, Cm
 * [requests, G, N]; `state` [num_states, D, N] fp32 (16-byte aligned) updated in place;
 * state_indices as in kda_step.
 */
typedef struct {
    const float *skip, *delta_bias;
    const void *z;
    const float *initial_state;
    float *final_state;
    void *saved;
    size_t saved_bytes;
    const int *cu_seqlens;
    int num_seqs;
    int zero_rest;
    int plain_delta;
    long long u_stride, delta_stride, z_stride, B_stride, C_stride, y_stride;
    void *workspace;
    size_t workspace_bytes;
} kda_scan_fwd_opts_t;

size_t kda_scan_saved_bytes(int B, int T, int D, int N, int num_seqs);
size_t kda_scan_fwd_workspace_bytes(int B, int T, int D, int N, int G, int num_seqs);

kda_status_t kda_scan_fwd(const void *u, const void *delta, const float *A, const void *Bm,
                          const void *Cm, void *y, int B, int T, int D, int N, int G, int dtype,
                          const kda_scan_fwd_opts_t *opts, kda_stream_t stream);

typedef struct {
    const float *skip, *delta_bias;
    const void *z;
    float *dskip, *ddelta_bias;
    void *dz;
    const float *d_final_state;
    float *d_initial_state;
    const void *saved;
    size_t saved_bytes;
    const int *cu_seqlens;
    int num_seqs;
    int zero_rest;
    int plain_delta;
    long long dy_stride, u_stride, delta_stride, z_stride, B_stride, C_stride;
    void *workspace;
    size_t workspace_bytes;
} kda_scan_bwd_opts_t;

size_t kda_scan_bwd_workspace_bytes(int B, int T, int D, int N, int G, int num_seqs);

kda_status_t kda_scan_bwd(const void *dy, const void *u, const void *delta, const float *A,
                          const void *Bm, const void *Cm, void *du, void *ddelta, float *dA, void *dB,
                          void *dC, int B, int T, int D, int N, int G, int dtype,
                          const kda_scan_bwd_opts_t *opts, kda_stream_t stream);

typedef struct {
    const float *skip, *delta_bias;
    const void *z;
    const int *state_indices;
    int num_states; /* 0 means requests */
    int plain_delta;
    long long u_stride, delta_stride, z_stride, B_stride, C_stride, y_stride;
} kda_scan_step_opts_t;

kda_status_t kda_scan_step(const void *u, const void *delta, const float *A, const void *Bm,
                           const void *Cm, float *state, void *y, int requests, int D, int N, int G,
                           int dtype, const kda_scan_step_opts_t *opts, kda_stream_t stream);

/*
 * Matrix product with its epilogue: y = act(x weight^T + bias) + residual, x [M, K], weight [N, K], y,
 * residual [M, N], bias [N], all KDA_BF16 or all KDA_FP16, with a row stride each (0 = width); bias
 * and residual may be NULL.  Sums are FP32 and rounded once, behind the residual.  `saved` [M, N]
 * (contiguous, of the type; NULL when no backward follows or without an activation) gets x weight^T +
 * bias, rounded.  Rows on 16-byte boundaries are taken as they are; of x and weight others are
 * copied to such boundaries first: kda_linear_copies() tells which, and `workspace`
 * (256-byte aligned) holds kda_linear_fwd_workspace_bytes() of that.
 *
 * Backward: dpre = dy act'(saved), rounded to the type as the operand of two products; dx = dpre
 * weight, dweight = dpre^T x [N, K], dbias = dpre's column sums (before the rounding), each rounded once
 * from FP32 sums in a fixed order; NULL = not wanted.  residual's gradient is dy itself.  `wanted` says
 * which (KDA_GRAD_*), as the pointers do.  So the derivative is taken at a rounded place and dx and dweight are products of a rounded
 * dpre: with an activation their error is some 1.4 times that of a result that is rounded once.
 */
#define KDA_COPY_X 1
#define KDA_COPY_WEIGHT 2
#define KDA_COPY_DY 4
#define KDA_GRAD_X 1
#define KDA_GRAD_WEIGHT 2
#define KDA_GRAD_BIAS 4

typedef struct {
    const void *bias, *residual;
    void *saved;
    int activation;
    long long x_stride, weight_stride, residual_stride, y_stride;
    void *workspace;
    size_t workspace_bytes;
} kda_linear_fwd_opts_t;

int kda_linear_copies(const void *x, long long x_stride, const void *weight, long long weight_stride,
                      const void *dy, long long dy_stride);
size_t kda_linear_fwd_workspace_bytes(int M, int K, int N, int copies);

kda_status_t kda_linear_fwd(const void *x, const void *weight, void *y, int M, int K, int N, int dtype,
                            const kda_linear_fwd_opts_t *opts, kda_stream_t stream);

typedef struct {
    const void *saved;
    int activation;
    long long dy_stride, x_stride, weight_stride, dx_stride;
    void *workspace;
    size_t workspace_bytes;
} kda_linear_bwd_opts_t;

size_t kda_linear_bwd_workspace_bytes(int M, int K, int N, int activation, int copies, int wanted);

kda_status_t kda_linear_bwd(const void *dy, const void *x, const void *weight, void *dx, void *dweight,
                            void *dbias, int M, int K, int N, int dtype,
                            const kda_linear_bwd_opts_t *opts, kda_stream_t stream);

/* Human-readable name of a status code (static storage, never NULL). */
const char *kda_status_str(kda_status_t status);

/*
 * Bounds-checked debug build.  The same sources compiled with -DKDA_DEBUG_CHECKS (the
 * build script's libkda_debug.so) check every global index their kernels compute
 * (output stores, incoming-gradient and beta reads, chunk-table reads; of the recurrence
 * and layer norm the tokens and rows that are read, states, and the slots of saved and
 * workspace buffers too) against the extent of its buffer.  An index out of range sets
 * KDA_DBG_STORE or KDA_DBG_LOAD in a caller-owned device word and the access is skipped;
 * a bounded wait that gives up sets KDA_DBG_WAIT.  Where the caller has set KDA_DBG_SHORT in the
 * word, every extent of the convolution, the scan and the matrix product counts as one less: the checks
 * of a buffer's last element or row then report and skip it, which shows that they are there.  Nothing traps or asserts.  TMA tiles
 * need no check: the tensor maps clip them.
 *
 * kda_debug_checks() is 1 in such a build, 0 otherwise.  kda_debug_set_flags(word)
 * makes every later launch of this library report into `word` (device memory, 4 bytes,
 * caller-owned; NULL stops reporting); the library never clears it.  Set it
 * before launching, from one thread.  Returns KDA_ERR_OPTION in a build without checks
 * and KDA_ERR_ALIGN for a word that is not 4-byte aligned.
 */
#define KDA_DBG_STORE 1u
#define KDA_DBG_LOAD 2u
#define KDA_DBG_WAIT 4u
#define KDA_DBG_SHORT 8u
int kda_debug_checks(void);
kda_status_t kda_debug_set_flags(unsigned int *device_word);

/*
 * In such a build, with `on` other than 0, the matrix product's waits on copies and products give up
 * at once, to see what a stalled pipeline leaves (kernels of up to 16 rows and a short contraction
 * have no such waits).  Waits for copies in flight at a kernel's end are not shortened.
 * KDA_ERR_OPTION in a build without checks.
 */
kda_status_t kda_debug_set_give_up(int on);

/* KDA_ABI_VERSION of the loaded library. */
int kda_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
