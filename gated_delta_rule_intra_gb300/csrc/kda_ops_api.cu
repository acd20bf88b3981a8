// C ABI of the recurrence, single-token and layer-norm operators: argument validation and
// dispatch (see include/kda.h).
#include <stdint.h>
#include <string.h>

#include <cuda_runtime.h>

#include "kda_ops.h"

#pragma GCC visibility push(default)
#include "kda.h"
#pragma GCC visibility pop

namespace kda {
kda_status_t require_device();  // kda_api.cu
unsigned *debug_flags();
}  // namespace kda

namespace {

// Bytes that a call reads or writes: one run, or rows of `row` bytes `step` apart.
struct Range {
    uintptr_t lo, hi, row, step;
    Range(const void *p, size_t bytes)
        : lo((uintptr_t)p), hi(p ? (uintptr_t)p + bytes : 0), row(bytes), step(bytes) {}
    Range(const void *p, long long rows, int width, long long stride, int es)
        : Range(p, rows ? ((size_t)(rows - 1) * stride + width) * es : 0) {
        row = (size_t)width * es;
        step = (size_t)stride * es;
    }
};

bool meet(const Range &a, const Range &b) {
    if (!(a.lo < b.hi && b.lo < a.hi)) return false;
    if (a.step != b.step) return true;
    // rows equally far apart may lie between each other's (column slices of one buffer)
    const uintptr_t off = b.lo >= a.lo ? (b.lo - a.lo) % a.step
                                       : (a.step - (a.lo - b.lo) % a.step) % a.step;
    return !(off >= a.row && off + b.row <= a.step);
}

// Every output against every input and every other output.
template <size_t NO, size_t NI> bool overlap(const Range (&out)[NO], const Range (&in)[NI]) {
    for (size_t o = 0; o < NO; ++o) {
        for (const Range &r : in)
            if (meet(out[o], r)) return true;
        for (size_t p = o + 1; p < NO; ++p)
            if (meet(out[o], out[p])) return true;
    }
    return false;
}

template <size_t N> bool misaligned(const void *const (&ps)[N], unsigned to) {
    for (const void *p : ps)
        if ((uintptr_t)p % to) return true;
    return false;
}

kda_status_t finish(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// What the forward saves, and the backward's workspace, for 64 tokens of a head: the state (or
// its gradient), e (or Y), the steps' tiles; FP16 with scales in BF16 training (kda_fast.cuh),
// BF16 hi and lo otherwise.
struct SlotBytes {
    size_t state, rows, tiles, scales;
    size_t saved() const { return state + rows + tiles + scales; }
    size_t work() const { return state + rows + scales; }
};
constexpr SlotBytes kFull = {65536, 32768, 8192, 0}, kFast = {32768, 16384, 8192, 160};

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// 64-token slots of a call (see seq_of() in kda_chunk.cuh).
long long chunk_slots(int B, int T, int num_seqs) {
    return num_seqs > 0 ? (long long)T / KDA_BT + num_seqs + 1
                        : (long long)B * (((long long)T + KDA_BT - 1) / KDA_BT);
}

kda_status_t check_chunk_shape(int B, int T, int H, int HV, bool varlen, int num_seqs) {
    if (B <= 0 || T < 0 || H <= 0 || HV <= 0 || HV > KDA_MAX_H || HV % H) return KDA_ERR_SHAPE;
    if (varlen && (B != 1 || num_seqs <= 0)) return KDA_ERR_SHAPE;
    if (!varlen && num_seqs != 0) return KDA_ERR_SHAPE;
    const long long seqs = varlen ? num_seqs : B;
    if (seqs * HV * 8 > 0x7fffffffLL) return KDA_ERR_SHAPE;  // grid limit
    if ((long long)B * T > 0x7fffffffLL - KDA_BT) return KDA_ERR_SHAPE;
    if ((long long)B * T * HV > (1LL << 52) / KDA_K) return KDA_ERR_SHAPE;
    if (chunk_slots(B, T, num_seqs) * HV > 0x7fffffffLL) return KDA_ERR_SHAPE;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_chunk_saved_bytes(int B, int T, int HV, int num_seqs, kda_dtype_t dtype,
                             int with_state) {
    if (check_chunk_shape(B, T, 1, HV, num_seqs > 0, num_seqs) != KDA_OK) return 0;
    const SlotBytes &s = dtype == KDA_BF16 && !with_state ? kFast : kFull;
    return up256((size_t)chunk_slots(B, T, num_seqs) * HV * s.saved());
}

kda_status_t kda_chunk_fwd(const void *q, const void *k, const void *v, const float *gate,
                           const float *beta, void *o, int B, int T, int H, kda_dtype_t dtype,
                           const kda_chunk_fwd_opts_t *opts, kda_stream_t stream) {
    kda_chunk_fwd_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    if (T > 0 && (!q || !k || !v || !gate || !beta || !o)) return KDA_ERR_NULL;
    const int HV = op.HV ? op.HV : H;
    const bool varlen = op.cu_seqlens != nullptr;
    kda_status_t st = check_chunk_shape(B, T, H, HV, varlen, op.num_seqs);
    if (st != KDA_OK) return st;
    if (dtype != KDA_BF16 && dtype != KDA_FP16) return KDA_ERR_DTYPE;
    const void *a16[] = {q, k, v, gate, o, op.initial_state, op.final_state};
    const void *a4[] = {beta, op.cu_seqlens};
    const void *a256[] = {op.saved};
    if (misaligned(a16, 16) || misaligned(a4, 4) || misaligned(a256, 256)) return KDA_ERR_ALIGN;
    const bool with_state = op.initial_state || op.final_state;
    bool fast = dtype == KDA_BF16 && !with_state;
    size_t saved = kda_chunk_saved_bytes(B, T, HV, op.num_seqs, dtype, with_state);
    if (op.saved && op.saved_bytes != saved && fast) {  // the caller's choice of the other kernels
        fast = false;
        saved = kda_chunk_saved_bytes(B, T, HV, op.num_seqs, dtype, 1);
    }
    if (op.saved && op.saved_bytes != saved) return KDA_ERR_WORKSPACE;
    const size_t rq = (size_t)B * T * H, rv = (size_t)B * T * HV;
    const int seqs = varlen ? op.num_seqs : B;
    const size_t states = (size_t)seqs * HV * KDA_K * KDA_K * 4;
    const Range in[] = {{q, rq * KDA_K * 2}, {k, rq * KDA_K * 2}, {v, rv * KDA_K * 2},
                        {gate, rv * KDA_K * 4}, {beta, rv * 4}, {op.initial_state, states},
                        {op.cu_seqlens, varlen ? ((size_t)seqs + 1) * 4 : 0}};
    const Range out[] = {{o, rv * KDA_K * 2}, {op.final_state, states}, {op.saved, saved}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (T == 0 && !op.final_state) return KDA_OK;
    if (varlen && op.zero_rest) {
        const kda::ZeroArgs z = {{o}, {(size_t)HV * KDA_K * 2}, 1, T, seqs, op.cu_seqlens, kda::debug_flags()};
        const cudaError_t e = kda::launch_zero_rest(z, (cudaStream_t)stream);
        if (e != cudaSuccess) return finish(e);
    }
    kda::ChunkFwdArgs a = {};
    a.q = q; a.k = k; a.v = v; a.gate = gate; a.beta = beta; a.o = o;
    a.initial_state = op.initial_state;
    a.final_state = op.final_state;
    if (op.saved) {
        const size_t n = (size_t)chunk_slots(B, T, op.num_seqs) * HV;
        const SlotBytes &s = fast ? kFast : kFull;
        a.ckpt = (char *)op.saved;
        a.e = a.ckpt + n * s.state;
        a.tiles = a.e + n * s.rows;
        a.scales = (float *)(a.tiles + n * s.tiles);
    }
    a.fast = fast;
    a.T = T; a.H = H; a.HV = HV; a.num_seqs = seqs;
    a.cu_seqlens = op.cu_seqlens;
    a.scale = op.scale != 0.f ? op.scale : 0.08838834764831845f;
    a.fp16 = dtype == KDA_FP16;
    a.rows_o = rv;
    a.units = (size_t)chunk_slots(B, T, op.num_seqs) * HV;
    a.states = states / 4;
    a.dbg = kda::debug_flags();
    return finish(kda::launch_chunk_fwd(a, (cudaStream_t)stream));
}

// The mode that wrote `saved_bytes`: 0 with states or FP16, 1 BF16 training, -1 neither.
static int saved_mode(int B, int T, int HV, int num_seqs, kda_dtype_t dtype, size_t saved_bytes) {
    if (saved_bytes && dtype == KDA_BF16 &&
        saved_bytes == kda_chunk_saved_bytes(B, T, HV, num_seqs, dtype, 0))
        return 1;
    return saved_bytes == kda_chunk_saved_bytes(B, T, HV, num_seqs, dtype, 1) ? 0 : -1;
}

size_t kda_chunk_bwd_workspace_bytes(int B, int T, int H, int HV, int num_seqs,
                                     kda_dtype_t dtype, size_t saved_bytes) {
    if (check_chunk_shape(B, T, H, HV, num_seqs > 0, num_seqs) != KDA_OK) return 0;
    const int mode = saved_mode(B, T, HV, num_seqs, dtype, saved_bytes);
    if (mode < 0) return 0;
    const size_t units = (size_t)chunk_slots(B, T, num_seqs) * HV;
    const size_t heads = HV > H ? (size_t)B * T * HV * KDA_K * 4 * 2 : 0;
    return up256(units * (mode ? kFast : kFull).work()) + heads;
}

kda_status_t kda_chunk_bwd(const void *q, const void *k, const float *gate, const float *beta,
                           const void *dout, void *dq, void *dk, void *dv, void *dgate,
                           void *dbeta, int B, int T, int H, kda_dtype_t dtype,
                           const kda_chunk_bwd_opts_t *opts, kda_stream_t stream) {
    if (!opts) return KDA_ERR_WORKSPACE;
    const kda_chunk_bwd_opts_t op = *opts;
    if (T > 0 && (!q || !k || !gate || !beta || !dout || !dq || !dk || !dv || !dgate || !dbeta))
        return KDA_ERR_NULL;
    const int HV = op.HV ? op.HV : H;
    const bool varlen = op.cu_seqlens != nullptr;
    kda_status_t st = check_chunk_shape(B, T, H, HV, varlen, op.num_seqs);
    if (st != KDA_OK) return st;
    if (dtype != KDA_BF16 && dtype != KDA_FP16) return KDA_ERR_DTYPE;
    const void *a16[] = {q, k, gate, dout, dq, dk, dv, dgate, op.d_final_state,
                         op.d_initial_state};
    const bool zero_rest = op.zero_rest & 1, gates32 = op.zero_rest & KDA_GATE_GRADS_FP32;
    const size_t gs = gates32 ? 4 : 2;  // bytes of an element of dgate and dbeta
    const void *a4[] = {beta, op.cu_seqlens}, *ab[] = {dbeta};
    const void *a256[] = {op.saved, op.workspace};
    if (misaligned(a16, 16) || misaligned(a4, 4) || misaligned(ab, (unsigned)gs) ||
        misaligned(a256, 256))
        return KDA_ERR_ALIGN;
    const int mode = saved_mode(B, T, HV, op.num_seqs, dtype, op.saved_bytes);
    if (mode < 0) return KDA_ERR_WORKSPACE;
    const size_t saved = op.saved_bytes;
    const size_t work =
        kda_chunk_bwd_workspace_bytes(B, T, H, HV, op.num_seqs, dtype, op.saved_bytes);
    if ((saved && !op.saved) ||
        (work && (!op.workspace || op.workspace_bytes < work)))
        return KDA_ERR_WORKSPACE;
    const size_t rq = (size_t)B * T * H, rv = (size_t)B * T * HV;
    const int seqs = varlen ? op.num_seqs : B;
    const size_t states = (size_t)seqs * HV * KDA_K * KDA_K * 4;
    const Range in[] = {{q, rq * KDA_K * 2}, {k, rq * KDA_K * 2}, {dout, rv * KDA_K * 2},
                        {gate, rv * KDA_K * 4}, {beta, rv * 4}, {op.d_final_state, states},
                        {op.cu_seqlens, varlen ? ((size_t)seqs + 1) * 4 : 0}, {op.saved, saved}};
    const Range out[] = {{dq, rq * KDA_K * 2}, {dk, rq * KDA_K * 2}, {dv, rv * KDA_K * 2},
                         {dgate, rv * KDA_K * gs}, {dbeta, rv * gs}, {op.d_initial_state, states},
                         {op.workspace, work}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (T == 0 && !op.d_initial_state) return KDA_OK;
    if (varlen && zero_rest) {
        const size_t head = KDA_K * 2;
        const kda::ZeroArgs z = {{dq, dk, dv, dgate, dbeta},
                                 {H * head, H * head, HV * head, HV * KDA_K * gs, HV * gs},
                                 5, T, seqs, op.cu_seqlens, kda::debug_flags()};
        const cudaError_t e = kda::launch_zero_rest(z, (cudaStream_t)stream);
        if (e != cudaSuccess) return finish(e);
    }
    kda::ChunkBwdArgs a = {};
    a.q = q; a.k = k; a.dout = dout; a.gate = gate; a.beta = beta;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dgate = dgate; a.dbeta = dbeta;
    a.d_final_state = op.d_final_state;
    a.d_initial_state = op.d_initial_state;
    const long long slots = chunk_slots(B, T, op.num_seqs);
    const size_t n = (size_t)slots * HV;
    a.fast = mode == 1;
    const SlotBytes &s = a.fast ? kFast : kFull;
    a.ckpt = (const char *)op.saved;
    a.e = a.ckpt + n * s.state;
    a.tiles = a.e + n * s.rows;
    a.scales = (const float *)(a.tiles + n * s.tiles);
    a.dckpt = (char *)op.workspace;
    a.y = a.dckpt + n * s.state;
    a.dscales = (float *)(a.y + n * s.rows);
    if (HV > H) {
        a.dq_hv = (float *)((char *)op.workspace + up256(n * s.work()));
        a.dk_hv = a.dq_hv + rv * KDA_K;
    }
    a.gates32 = gates32;
    a.B = B; a.T = T; a.H = H; a.HV = HV; a.num_seqs = seqs;
    a.slots = (int)slots;
    a.cu_seqlens = op.cu_seqlens;
    a.scale = op.scale != 0.f ? op.scale : 0.08838834764831845f;
    a.fp16 = dtype == KDA_FP16;
    a.rows_o = rv;
    a.units = n;
    a.states = states / 4;
    a.dbg = kda::debug_flags();
    return finish(kda::launch_chunk_bwd(a, (cudaStream_t)stream));
}

kda_status_t kda_step(const void *q, const void *k, const void *v, const float *gate,
                      const float *beta, float *state, void *o, int N, int H, kda_dtype_t dtype,
                      const kda_step_opts_t *opts, kda_stream_t stream) {
    kda_step_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    const int HV = op.HV ? op.HV : H;
    if (N < 0 || H <= 0 || HV <= 0 || HV > KDA_MAX_H || HV % H) return KDA_ERR_SHAPE;
    if (op.num_states < 0 || (long long)N * HV * 4 > 0x7fffffffLL) return KDA_ERR_SHAPE;
    const int states = op.num_states ? op.num_states : N;
    if (!op.state_indices && states < N) return KDA_ERR_SHAPE;
    if (N > 0 && (!q || !k || !v || !gate || !beta || !state || !o)) return KDA_ERR_NULL;
    if (dtype != KDA_BF16 && dtype != KDA_FP16) return KDA_ERR_DTYPE;
    const void *a16[] = {q, k, v, gate, state, o};
    const void *a4[] = {beta, op.state_indices};
    if (misaligned(a16, 16) || misaligned(a4, 4)) return KDA_ERR_ALIGN;
    const size_t rq = (size_t)N * H, rv = (size_t)N * HV;
    const Range in[] = {{q, rq * KDA_K * 2}, {k, rq * KDA_K * 2}, {v, rv * KDA_K * 2},
                        {gate, rv * KDA_K * 4}, {beta, rv * 4},
                        {op.state_indices, (size_t)N * 4}};
    const Range out[] = {{o, rv * KDA_K * 2}, {state, (size_t)states * HV * KDA_K * KDA_K * 4}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    kda_status_t st = kda::require_device();
    if (st != KDA_OK) return st;
    (void)cudaGetLastError();
    if (N == 0) return KDA_OK;
    kda::StepArgs a = {};
    a.q = q; a.k = k; a.v = v; a.gate = gate; a.beta = beta; a.state = state; a.o = o;
    a.N = N; a.H = H; a.HV = HV;
    a.state_indices = op.state_indices;
    a.num_states = states;
    a.scale = op.scale != 0.f ? op.scale : 0.08838834764831845f;
    a.fp16 = dtype == KDA_FP16;
    a.dbg = kda::debug_flags();
    return finish(kda::launch_step(a, (cudaStream_t)stream));
}

static kda_status_t check_norm(long long rows, int width, int dtype, int wdtype) {
    if (rows < 0 || width <= 0 || rows > (1LL << 52) / width) return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16 && dtype != KDA_FP16 && dtype != KDA_FP32) return KDA_ERR_DTYPE;
    if (wdtype != dtype && wdtype != KDA_FP32) return KDA_ERR_DTYPE;
    return KDA_OK;
}

kda_status_t kda_layer_norm_fwd(const void *x, const void *weight, const void *bias, void *y,
                                float *mean, float *rstd, long long rows, int width, float eps,
                                int dtype, int wdtype, long long x_stride, long long y_stride,
                                kda_stream_t stream) {
    kda_status_t st = check_norm(rows, width, dtype, wdtype);
    if (st != KDA_OK) return st;
    if (rows > 0 && (!x || !y)) return KDA_ERR_NULL;
    if (!x_stride) x_stride = width;
    if (!y_stride) y_stride = width;
    if (x_stride < width || y_stride < width) return KDA_ERR_SHAPE;
    const int es = dtype == KDA_FP32 ? 4 : 2, ws = wdtype == KDA_FP32 ? 4 : 2;
    const void *ae[] = {x, y}, *aw[] = {weight, bias}, *a4[] = {mean, rstd};
    if (misaligned(ae, es) || misaligned(aw, ws) || misaligned(a4, 4)) return KDA_ERR_ALIGN;
    const Range in[] = {{x, rows, width, x_stride, es}, {weight, (size_t)width * ws},
                        {bias, (size_t)width * ws}};
    const Range out[] = {{y, rows, width, y_stride, es}, {mean, (size_t)rows * 4},
                         {rstd, (size_t)rows * 4}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (rows == 0) return KDA_OK;
    kda::NormArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.rows = rows; a.width = width; a.dtype = dtype; a.wdtype = wdtype;
    a.x_stride = x_stride; a.y_stride = y_stride;
    a.eps = eps;
    a.dbg = kda::debug_flags();
    return finish(kda::launch_norm_fwd(a, (cudaStream_t)stream));
}

size_t kda_layer_norm_bwd_workspace_bytes(long long rows, int width) {
    if (check_norm(rows, width, KDA_FP32, KDA_FP32) != KDA_OK) return 0;
    return (size_t)kda::norm_bwd_ctas(rows, width) * 2 * width * 4;
}

kda_status_t kda_layer_norm_bwd(const void *dy, const void *x, const void *weight,
                                const float *mean, const float *rstd, void *dx, float *dweight,
                                float *dbias, long long rows, int width, int dtype, int wdtype,
                                long long dy_stride, long long x_stride, long long dx_stride,
                                void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda_status_t st = check_norm(rows, width, dtype, wdtype);
    if (st != KDA_OK) return st;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return KDA_ERR_NULL;
    if (!dweight != !dbias) return KDA_ERR_NULL;
    if (!x_stride) x_stride = width;
    if (!dy_stride) dy_stride = width;
    if (!dx_stride) dx_stride = width;
    if (x_stride < width || dy_stride < width || dx_stride < width) return KDA_ERR_SHAPE;
    const int es = dtype == KDA_FP32 ? 4 : 2, ws = wdtype == KDA_FP32 ? 4 : 2;
    const void *ae[] = {dy, x, dx}, *aw[] = {weight}, *a4[] = {mean, rstd, dweight, dbias},
               *a16[] = {workspace};
    if (misaligned(ae, es) || misaligned(aw, ws) || misaligned(a4, 4) || misaligned(a16, 16))
        return KDA_ERR_ALIGN;
    const size_t need = dweight ? kda_layer_norm_bwd_workspace_bytes(rows, width) : 0;
    if (need && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const Range in[] = {{dy, rows, width, dy_stride, es}, {x, rows, width, x_stride, es},
                        {weight, (size_t)width * ws},
                        {mean, (size_t)rows * 4}, {rstd, (size_t)rows * 4}};
    const Range out[] = {{dx, rows, width, dx_stride, es}, {dweight, (size_t)width * 4},
                         {dbias, (size_t)width * 4}, {need ? workspace : nullptr, need}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (rows == 0 && !dweight) return KDA_OK;
    kda::NormArgs a = {};
    a.x = x; a.weight = weight; a.dy = dy; a.dx = dx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dweight = dweight; a.dbias = dbias; a.partial = (float *)workspace;
    a.rows = rows; a.width = width; a.dtype = dtype; a.wdtype = wdtype;
    a.x_stride = x_stride; a.dy_stride = dy_stride; a.dx_stride = dx_stride;
    a.partials = kda::norm_bwd_ctas(rows, width);
    a.dbg = kda::debug_flags();
    return finish(kda::launch_norm_bwd(a, (cudaStream_t)stream));
}

}  // extern "C"
