// C ABI of the short convolution, the selective scan and the matrix product with its epilogue:
// argument validation and dispatch (see include/kda.h).
#include <string.h>

#include "kda_check.h"
#include "kda_layer.h"

namespace {

using kda::finish;
using kda::misaligned;
using kda::overlap;
using kda::Range;
using kda::Tokens;
using kda::up256;

kda_status_t check_tokens(int B, int T, const int *cu, int num_seqs, Tokens &tok) {
    if (B <= 0 || T < 0 || num_seqs < 0) return KDA_ERR_SHAPE;
    if (cu ? B != 1 || num_seqs == 0 : num_seqs != 0) return KDA_ERR_SHAPE;
    if ((long long)B * T > 0x7fffffffLL - 4096) return KDA_ERR_SHAPE;
    tok.B = B;
    tok.T = T;
    tok.num_seqs = cu ? num_seqs : B;
    tok.cu_seqlens = cu;
    return KDA_OK;
}
bool any_type(int t) { return t == KDA_BF16 || t == KDA_FP16 || t == KDA_FP32; }
// Rows of `width` elements, stride apart (0: width).
bool stride_ok(long long &stride, long long width) {
    if (!stride) stride = width;
    return stride >= width && stride <= (1LL << 40);
}
// Zeros for tokens in no sequence.
struct Out {
    void *p;
    size_t row;
};
template <size_t N>
cudaError_t zero_rest(const Tokens &tok, const Out (&outs)[N], kda_stream_t stream) {
    kda::ZeroArgs z = {};
    for (const Out &o : outs)
        if (o.p) {
            z.out[z.count] = o.p;
            z.row[z.count++] = o.row;
        }
    z.T = tok.T;
    z.num_seqs = tok.num_seqs;
    z.cu_seqlens = tok.cu_seqlens;
    z.dbg = kda::debug_flags();
    return kda::launch_zero_rest(z, (cudaStream_t)stream);
}
size_t cu_bytes(const Tokens &t) { return t.cu_seqlens ? ((size_t)t.num_seqs + 1) * 4 : 0; }

// ---------------------------------------------------------------- convolution
kda_status_t check_conv(int D, int W, int dtype, int wdtype, int act) {
    if (D <= 0 || D > (1 << 28) || W < 2 || W > 4) return KDA_ERR_SHAPE;
    if (!any_type(dtype) || (wdtype != dtype && wdtype != KDA_FP32)) return KDA_ERR_DTYPE;
    if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return KDA_ERR_OPTION;
    return KDA_OK;
}
bool grid_ok(long long ctas) { return ctas <= 0x7fffffffLL; }
kda::ConvArgs conv_args(const void *x, const void *weight, const void *bias, int D, int W, int dtype,
                        int wdtype, int act) {
    kda::ConvArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias;
    a.D = D; a.W = W; a.dtype = dtype; a.wdtype = wdtype; a.act = act;
    a.dbg = kda::debug_flags();
    return a;
}

// ---------------------------------------------------------------- scan
kda_status_t check_scan(int D, int N, int G, int dtype) {
    if (D <= 0 || D > (1 << 28) || N <= 0 || N > kda::kScanMaxN || G <= 0 || D % G) return KDA_ERR_SHAPE;
    if ((long long)G * N > (1 << 28)) return KDA_ERR_SHAPE;  // rows of B and C are counted in 32 bits
    return any_type(dtype) ? KDA_OK : KDA_ERR_DTYPE;
}
kda_status_t scan_shape(int B, int T, int D, int N, int G, int num_seqs, Tokens &tok) {
    static const int some = 0;
    kda_status_t st = check_tokens(B, T, num_seqs ? &some : nullptr, num_seqs, tok);
    if (st == KDA_OK) st = check_scan(D, N, G, KDA_FP32);
    if (st != KDA_OK) return st;
    if (tok.pieces(kda::kScanTile) > (1LL << 52) / ((long long)D * 64)) return KDA_ERR_SHAPE;
    return grid_ok(tok.pieces(kda::kScanTile) * kda::scan_blocks(D, N, G)) ? KDA_OK : KDA_ERR_SHAPE;
}
size_t scan_saved_floats(const Tokens &t, int D, int N) {
    return 2 * (size_t)t.pieces(kda::kScanTile) * D * kda::scan_padded(N);
}
size_t scan_saved_bytes(const Tokens &t, int D, int N) {  // and y before the gate
    return up256(scan_saved_floats(t, D, N) * 4) + up256((size_t)t.rows() * (((size_t)D + 3) / 4 * 16));
}
// Floats of the first pass over segments; 0 where every sequence is one segment.
struct Segments {
    int size;
    size_t slots, ends, sums;
    Segments(const Tokens &t, int D, int N, int G, bool back) {
        size = kda::scan_segment(t, D, N, G, back);
        slots = (size_t)t.pieces(size);
        const bool cut = t.T > size;
        ends = cut ? slots * D * kda::scan_padded(N) : 0;
        sums = cut ? slots * D : 0;
    }
};

// ---------------------------------------------------------------- matrix product
kda_status_t check_linear(int M, int K, int N, int dtype, int act) {
    if (M < 0 || K <= 0 || N <= 0 || M > (1 << 30) || K > (1 << 24) || N > (1 << 24)) return KDA_ERR_SHAPE;
    // every tensor below 2^40 elements, every product's tiles a 32-bit number
    auto tiles = [](long long m, long long n) { return ((m + 127) / 128) * ((n + 63) / 64); };
    if ((long long)M * K > (1LL << 40) || (long long)M * N > (1LL << 40) || (long long)N * K > (1LL << 40) ||
        !(tiles(M, N) < 1 << 26 && tiles(M, K) < 1 << 26 && tiles(N, K) < 1 << 26))
        return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16 && dtype != KDA_FP16) return KDA_ERR_DTYPE;
    return act >= KDA_ACT_NONE && act <= KDA_ACT_RELU ? KDA_OK : KDA_ERR_OPTION;
}
long long up8(long long n) { return (n + 7) / 8 * 8; }
// Rows that a tensor map takes as they are: on 16-byte boundaries.
bool rows_ok(const void *p, long long stride) { return (uintptr_t)p % 16 == 0 && stride % 8 == 0; }
size_t copy_bytes(long long rows, int width) { return up256((size_t)rows * up8(width) * 2); }

struct Work {  // parts of a workspace, one behind the other
    char *at;
    void *take(size_t bytes) {
        char *p = at;
        at += up256(bytes);
        return p;
    }
};
// Copies of the tensors that need them, in one launch.
struct Copies {
    kda::CopyArgs jobs[2];
    int count = 0;
    void add(const void *&p, long long &stride, long long rows, int width, Work &w) {
        if (rows_ok(p, stride)) return;
        const long long ld = up8(width);
        void *to = w.take((size_t)rows * ld * 2);
        jobs[count++] = {p, to, rows, stride, ld, width, kda::debug_flags()};
        p = to;
        stride = ld;
    }
    cudaError_t run(cudaStream_t stream) const {
        return count ? kda::launch_copy_rows(jobs[0], count > 1 ? jobs + 1 : nullptr, stream) : cudaSuccess;
    }
};

}  // namespace

extern "C" {

kda_status_t kda_conv_fwd(const void *x, const void *weight, const void *bias, void *y, int B, int T,
                          int D, int W, int dtype, int wdtype, int activation,
                          const kda_conv_fwd_opts_t *opts, kda_stream_t stream) {
    kda_conv_fwd_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    Tokens tok;
    kda_status_t st = check_tokens(B, T, op.cu_seqlens, op.num_seqs, tok);
    if (st == KDA_OK) st = check_conv(D, W, dtype, wdtype, activation);
    if (st != KDA_OK) return st;
    if (!weight || (T > 0 && (!x || !y))) return KDA_ERR_NULL;
    if (!stride_ok(op.x_stride, D) || !stride_ok(op.y_stride, D) || !grid_ok(tok.pieces(64) * ((D + 31) / 32)))
        return KDA_ERR_SHAPE;
    const int es = kda::esize(dtype), ws = kda::esize(wdtype);
    const void *ae[] = {x, y, op.initial_state, op.final_state}, *aw[] = {weight, bias}, *a4[] = {op.cu_seqlens};
    if (misaligned(ae, es) || misaligned(aw, ws) || misaligned(a4, 4)) return KDA_ERR_ALIGN;
    const size_t states = (size_t)tok.num_seqs * (W - 1) * D * es;
    const Range in[] = {{x, tok.rows(), D, op.x_stride, es}, {weight, (size_t)D * W * ws},
                        {bias, (size_t)D * ws}, {op.initial_state, states}, {op.cu_seqlens, cu_bytes(tok)}};
    const Range out[] = {{y, tok.rows(), D, op.y_stride, es}, {op.final_state, states}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (T == 0 && !op.final_state) return KDA_OK;
    if (op.zero_rest && tok.cu_seqlens) {
        if (op.y_stride != D) return KDA_ERR_OPTION;
        const cudaError_t e = zero_rest(tok, {Out{y, (size_t)D * es}}, stream);
        if (e != cudaSuccess) return finish(e);
    }
    kda::ConvArgs a = conv_args(x, weight, bias, D, W, dtype, wdtype, activation);
    a.tok = tok;
    a.y = y;
    a.initial = op.initial_state;
    a.final = op.final_state;
    a.x_stride = op.x_stride; a.y_stride = op.y_stride;
    return finish(kda::launch_conv_fwd(a, (cudaStream_t)stream));
}

size_t kda_conv_bwd_workspace_bytes(int B, int T, int D, int W, int num_seqs) {
    static const int some = 0;
    Tokens tok;
    if (check_tokens(B, T, num_seqs ? &some : nullptr, num_seqs, tok) != KDA_OK ||
        check_conv(D, W, KDA_FP32, KDA_FP32, 0) != KDA_OK)
        return 0;
    return (size_t)kda::conv_partials(tok.pieces(kda::kConvPiece), D) * (W + 1) * D * 4;
}

kda_status_t kda_conv_bwd(const void *dy, const void *x, const void *weight, const void *bias, void *dx,
                          float *dweight, float *dbias, int B, int T, int D, int W, int dtype, int wdtype,
                          int activation, const kda_conv_bwd_opts_t *opts, kda_stream_t stream) {
    kda_conv_bwd_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    Tokens tok;
    kda_status_t st = check_tokens(B, T, op.cu_seqlens, op.num_seqs, tok);
    if (st == KDA_OK) st = check_conv(D, W, dtype, wdtype, activation);
    if (st != KDA_OK) return st;
    if (!weight || (T > 0 && (!x || !dy || !dx)) || !dweight != !dbias) return KDA_ERR_NULL;
    if (!stride_ok(op.x_stride, D) || !stride_ok(op.dy_stride, D) || !stride_ok(op.dx_stride, D) ||
        !grid_ok(tok.pieces(64) * ((D + 31) / 32)))
        return KDA_ERR_SHAPE;
    const int es = kda::esize(dtype), ws = kda::esize(wdtype);
    const void *ae[] = {x, dy, dx, op.initial_state, op.d_final_state, op.d_initial_state};
    const void *aw[] = {weight, bias}, *a4[] = {op.cu_seqlens, dweight, dbias}, *a16[] = {op.workspace};
    if (misaligned(ae, es) || misaligned(aw, ws) || misaligned(a4, 4) || misaligned(a16, 16)) return KDA_ERR_ALIGN;
    const size_t need = dweight ? kda_conv_bwd_workspace_bytes(B, T, D, W, op.num_seqs) : 0;
    if (need && (!op.workspace || op.workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const size_t states = (size_t)tok.num_seqs * (W - 1) * D * es;
    const Range in[] = {{x, tok.rows(), D, op.x_stride, es}, {dy, tok.rows(), D, op.dy_stride, es},
                        {weight, (size_t)D * W * ws}, {bias, (size_t)D * ws}, {op.initial_state, states},
                        {op.d_final_state, states}, {op.cu_seqlens, cu_bytes(tok)}};
    const Range out[] = {{dx, tok.rows(), D, op.dx_stride, es}, {dweight, (size_t)D * W * 4},
                         {dbias, (size_t)D * 4}, {op.d_initial_state, states}, {need ? op.workspace : nullptr, need}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (T == 0 && !op.d_initial_state && !dweight) return KDA_OK;
    if (op.zero_rest && tok.cu_seqlens && T > 0) {
        if (op.dx_stride != D) return KDA_ERR_OPTION;
        const cudaError_t e = zero_rest(tok, {Out{dx, (size_t)D * es}}, stream);
        if (e != cudaSuccess) return finish(e);
    }
    kda::ConvArgs a = conv_args(x, weight, bias, D, W, dtype, wdtype, activation);
    a.tok = tok;
    a.dy = dy; a.dx = dx;
    a.initial = op.initial_state;
    a.d_final = op.d_final_state;
    a.d_initial = op.d_initial_state;
    a.dweight = dweight; a.dbias = dbias;
    a.partial = (float *)op.workspace;
    a.partials = kda::conv_partials(tok.pieces(kda::kConvPiece), D);
    a.partial_floats = need / 4;
    a.x_stride = op.x_stride; a.dy_stride = op.dy_stride; a.dx_stride = op.dx_stride;
    return finish(kda::launch_conv_bwd(a, (cudaStream_t)stream));
}

kda_status_t kda_conv_step(const void *x, const void *weight, const void *bias, void *state, void *y, int N,
                           int D, int W, int dtype, int wdtype, int activation,
                           const kda_conv_step_opts_t *opts, kda_stream_t stream) {
    kda_conv_step_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    kda_status_t st = check_conv(D, W, dtype, wdtype, activation);
    if (st != KDA_OK) return st;
    const int states = op.num_states ? op.num_states : N;
    if (N < 0 || N > 65535 || op.num_states < 0 || (!op.state_indices && states < N)) return KDA_ERR_SHAPE;
    if (!stride_ok(op.x_stride, D) || !stride_ok(op.y_stride, D)) return KDA_ERR_SHAPE;
    if (!weight || (N > 0 && (!x || !y || !state))) return KDA_ERR_NULL;
    const int es = kda::esize(dtype), ws = kda::esize(wdtype);
    const void *ae[] = {x, y, state}, *aw[] = {weight, bias}, *a4[] = {op.state_indices};
    if (misaligned(ae, es) || misaligned(aw, ws) || misaligned(a4, 4)) return KDA_ERR_ALIGN;
    const Range in[] = {{x, N, D, op.x_stride, es}, {weight, (size_t)D * W * ws}, {bias, (size_t)D * ws},
                        {op.state_indices, (size_t)N * 4}};
    const Range out[] = {{y, N, D, op.y_stride, es}, {state, (size_t)states * (W - 1) * D * es}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (N == 0) return KDA_OK;
    kda::ConvArgs a = conv_args(x, weight, bias, D, W, dtype, wdtype, activation);
    a.y = y;
    a.state = state;
    a.state_indices = op.state_indices;
    a.N = N;
    a.num_states = states;
    a.x_stride = op.x_stride; a.y_stride = op.y_stride;
    return finish(kda::launch_conv_step(a, (cudaStream_t)stream));
}

size_t kda_scan_saved_bytes(int B, int T, int D, int N, int num_seqs) {
    Tokens tok;
    if (scan_shape(B, T, D, N, 1, num_seqs, tok) != KDA_OK) return 0;
    return scan_saved_bytes(tok, D, N);
}

size_t kda_scan_fwd_workspace_bytes(int B, int T, int D, int N, int G, int num_seqs) {
    Tokens tok;
    if (scan_shape(B, T, D, N, G, num_seqs, tok) != KDA_OK) return 0;
    static const int some = 0;
    tok.cu_seqlens = num_seqs ? &some : nullptr;
    const Segments s(tok, D, N, G, false);
    return up256(s.ends * 4) + up256(s.sums * 4);
}

kda_status_t kda_scan_fwd(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                          void *y, int B, int T, int D, int N, int G, int dtype,
                          const kda_scan_fwd_opts_t *opts, kda_stream_t stream) {
    kda_scan_fwd_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    Tokens tok;
    kda_status_t st = check_tokens(B, T, op.cu_seqlens, op.num_seqs, tok);
    if (st == KDA_OK) st = scan_shape(B, T, D, N, G, op.num_seqs, tok);
    if (st != KDA_OK) return st;
    tok.cu_seqlens = op.cu_seqlens;
    if (!any_type(dtype)) return KDA_ERR_DTYPE;
    if (!A || (T > 0 && (!u || !delta || !Bm || !Cm || !y))) return KDA_ERR_NULL;
    if (!stride_ok(op.u_stride, D) || !stride_ok(op.delta_stride, D) || !stride_ok(op.z_stride, D) ||
        !stride_ok(op.y_stride, D) || !stride_ok(op.B_stride, (long long)G * N) ||
        !stride_ok(op.C_stride, (long long)G * N))
        return KDA_ERR_SHAPE;
    const int es = kda::esize(dtype);
    const void *ae[] = {u, delta, op.z, Bm, Cm, y};
    const void *a4[] = {A, op.skip, op.delta_bias, op.cu_seqlens, op.initial_state, op.final_state};
    const void *a256[] = {op.saved, op.workspace};
    if (misaligned(ae, es) || misaligned(a4, 4) || misaligned(a256, 256)) return KDA_ERR_ALIGN;
    const size_t saved = scan_saved_bytes(tok, D, N);
    const size_t need = kda_scan_fwd_workspace_bytes(B, T, D, N, G, op.num_seqs);
    if ((op.saved && op.saved_bytes != saved) || (need && (!op.workspace || op.workspace_bytes < need)))
        return KDA_ERR_WORKSPACE;
    const long long rows = tok.rows();
    const size_t states = (size_t)tok.num_seqs * D * N * 4, ds = (size_t)D * 4;
    const Range in[] = {{u, rows, D, op.u_stride, es}, {delta, rows, D, op.delta_stride, es},
                        {op.z, op.z ? rows : 0, D, op.z_stride, es}, {Bm, rows, G * N, op.B_stride, es},
                        {Cm, rows, G * N, op.C_stride, es}, {A, (size_t)D * N * 4}, {op.skip, ds},
                        {op.delta_bias, ds}, {op.initial_state, states}, {op.cu_seqlens, cu_bytes(tok)}};
    const Range out[] = {{y, rows, D, op.y_stride, es}, {op.final_state, states}, {op.saved, saved},
                         {need ? op.workspace : nullptr, need}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (T == 0 && !op.final_state) return KDA_OK;
    if (op.zero_rest && tok.cu_seqlens && T > 0) {
        if (op.y_stride != D) return KDA_ERR_OPTION;
        const cudaError_t e = zero_rest(tok, {Out{y, (size_t)D * es}}, stream);
        if (e != cudaSuccess) return finish(e);
    }
    const Segments s(tok, D, N, G, false);
    kda::ScanArgs a = {};
    a.tok = tok;
    a.u = u; a.delta = delta; a.z = op.z; a.B = Bm; a.C = Cm;
    a.A = A; a.skip = op.skip; a.delta_bias = op.delta_bias;
    a.y = y;
    a.initial = op.initial_state;
    a.final = op.final_state;
    a.saved = (float *)op.saved;
    if (op.saved && op.z) a.open = (float *)((char *)op.saved + up256(scan_saved_floats(tok, D, N) * 4));
    a.D = D; a.N = N; a.G = G; a.dtype = dtype;
    a.softplus = !op.plain_delta;
    a.u_stride = op.u_stride; a.delta_stride = op.delta_stride; a.z_stride = op.z_stride;
    a.B_stride = op.B_stride; a.C_stride = op.C_stride; a.y_stride = op.y_stride;
    a.segment = s.size;
    if (need) {
        a.ends = (float *)op.workspace;
        a.sums = (float *)((char *)op.workspace + up256(s.ends * 4));
    }
    a.saved_floats = scan_saved_floats(tok, D, N);
    a.open_floats = (size_t)rows * ((D + 3) / 4 * 4);
    a.segment_floats = s.ends;
    a.sum_floats = s.sums;
    a.dbg = kda::debug_flags();
    return finish(kda::launch_scan_fwd(a, (cudaStream_t)stream));
}

// ends, sums, part_A, part_D, part_bc
static size_t scan_bwd_work(const Tokens &tok, int D, int N, int G, const Segments &s, size_t (&part)[5]) {
    const int np = kda::scan_padded(N);
    part[0] = up256(s.ends * 4);
    part[1] = up256(s.sums * 4);
    part[2] = up256(s.slots * D * np * 4);
    part[3] = up256(s.slots * D * 2 * 4);
    part[4] = up256((size_t)tok.rows() * (size_t)kda::scan_blocks(D, N, G) * 2 * np * 4);
    return part[0] + part[1] + part[2] + part[3] + part[4];
}

size_t kda_scan_bwd_workspace_bytes(int B, int T, int D, int N, int G, int num_seqs) {
    Tokens tok;
    if (scan_shape(B, T, D, N, G, num_seqs, tok) != KDA_OK) return 0;
    static const int some = 0;
    tok.cu_seqlens = num_seqs ? &some : nullptr;
    size_t part[5];
    return scan_bwd_work(tok, D, N, G, Segments(tok, D, N, G, true), part);
}

kda_status_t kda_scan_bwd(const void *dy, const void *u, const void *delta, const float *A, const void *Bm,
                          const void *Cm, void *du, void *ddelta, float *dA, void *dB, void *dC, int B,
                          int T, int D, int N, int G, int dtype, const kda_scan_bwd_opts_t *opts,
                          kda_stream_t stream) {
    if (!opts) return KDA_ERR_WORKSPACE;
    kda_scan_bwd_opts_t op = *opts;
    Tokens tok;
    kda_status_t st = check_tokens(B, T, op.cu_seqlens, op.num_seqs, tok);
    if (st == KDA_OK) st = scan_shape(B, T, D, N, G, op.num_seqs, tok);
    if (st != KDA_OK) return st;
    tok.cu_seqlens = op.cu_seqlens;
    if (!any_type(dtype)) return KDA_ERR_DTYPE;
    if (!A || !dA || (T > 0 && (!dy || !u || !delta || !Bm || !Cm || !du || !ddelta || !dB || !dC)) ||
        !op.z != !op.dz || !op.skip != !op.dskip || !op.delta_bias != !op.ddelta_bias)
        return KDA_ERR_NULL;
    if (!stride_ok(op.u_stride, D) || !stride_ok(op.delta_stride, D) || !stride_ok(op.z_stride, D) ||
        !stride_ok(op.dy_stride, D) || !stride_ok(op.B_stride, (long long)G * N) ||
        !stride_ok(op.C_stride, (long long)G * N))
        return KDA_ERR_SHAPE;
    const int es = kda::esize(dtype);
    const void *ae[] = {dy, u, delta, op.z, Bm, Cm, du, ddelta, op.dz, dB, dC};
    const void *a4[] = {A, op.skip, op.delta_bias, op.cu_seqlens, dA, op.dskip, op.ddelta_bias,
                        op.d_final_state, op.d_initial_state};
    const void *a256[] = {op.saved, op.workspace};
    if (misaligned(ae, es) || misaligned(a4, 4) || misaligned(a256, 256)) return KDA_ERR_ALIGN;
    const Segments s(tok, D, N, G, true);
    size_t part[5];
    const size_t saved = scan_saved_bytes(tok, D, N);
    const size_t need = scan_bwd_work(tok, D, N, G, s, part);
    if (!op.saved || op.saved_bytes != saved || !op.workspace || op.workspace_bytes < need)
        return KDA_ERR_WORKSPACE;
    const long long rows = tok.rows();
    const size_t states = (size_t)tok.num_seqs * D * N * 4, ds = (size_t)D * 4;
    const size_t full = (size_t)rows * D * es, vec = (size_t)rows * G * N * es;
    const Range in[] = {{dy, rows, D, op.dy_stride, es}, {u, rows, D, op.u_stride, es},
                        {delta, rows, D, op.delta_stride, es}, {op.z, op.z ? rows : 0, D, op.z_stride, es},
                        {Bm, rows, G * N, op.B_stride, es}, {Cm, rows, G * N, op.C_stride, es},
                        {A, (size_t)D * N * 4}, {op.skip, ds}, {op.delta_bias, ds},
                        {op.d_final_state, states}, {op.cu_seqlens, cu_bytes(tok)}, {op.saved, saved}};
    const Range out[] = {{du, full}, {ddelta, full}, {op.dz, full}, {dB, vec}, {dC, vec},
                         {dA, (size_t)D * N * 4}, {op.dskip, ds}, {op.ddelta_bias, ds},
                         {op.d_initial_state, states}, {op.workspace, need}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (op.zero_rest && tok.cu_seqlens && T > 0) {
        const size_t row = (size_t)D * es, v = (size_t)G * N * es;
        const cudaError_t e = zero_rest(tok, {Out{du, row}, Out{ddelta, row}, Out{op.dz, row}, Out{dB, v},
                                              Out{dC, v}}, stream);
        if (e != cudaSuccess) return finish(e);
    }
    kda::ScanArgs a = {};
    a.tok = tok;
    a.u = u; a.delta = delta; a.z = op.z; a.B = Bm; a.C = Cm;
    a.A = A; a.skip = op.skip; a.delta_bias = op.delta_bias;
    a.saved = (float *)op.saved;
    if (op.saved && op.z) a.open = (float *)((char *)op.saved + up256(scan_saved_floats(tok, D, N) * 4));
    a.D = D; a.N = N; a.G = G; a.dtype = dtype;
    a.softplus = !op.plain_delta;
    a.u_stride = op.u_stride; a.delta_stride = op.delta_stride; a.z_stride = op.z_stride;
    a.B_stride = op.B_stride; a.C_stride = op.C_stride; a.dy_stride = op.dy_stride;
    a.du_stride = a.ddelta_stride = a.dz_stride = D;
    a.dy = dy; a.du = du; a.ddelta = ddelta; a.dz = op.dz; a.dB = dB; a.dC = dC;
    a.dA = dA; a.dskip = op.dskip; a.ddelta_bias = op.ddelta_bias;
    a.d_final = op.d_final_state;
    a.d_initial = op.d_initial_state;
    a.segment = s.size;
    char *at = (char *)op.workspace;
    if (s.ends) {
        a.ends = (float *)at;
        a.sums = (float *)(at + part[0]);
    }
    at += part[0] + part[1];
    a.part_A = (float *)at;
    a.part_D = (float *)(at + part[2]);
    a.part_bc = (float *)(at + part[2] + part[3]);
    a.saved_floats = scan_saved_floats(tok, D, N);
    a.open_floats = (size_t)rows * ((D + 3) / 4 * 4);
    a.segment_floats = s.slots * D * kda::scan_padded(N);
    a.sum_floats = s.sums;
    a.part_D_floats = s.slots * D * 2;
    a.part_bc_floats = (size_t)rows * (size_t)kda::scan_blocks(D, N, G) * 2 * kda::scan_padded(N);
    a.dbg = kda::debug_flags();
    return finish(kda::launch_scan_bwd(a, (cudaStream_t)stream));
}

kda_status_t kda_scan_step(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                           float *state, void *y, int requests, int D, int N, int G, int dtype,
                           const kda_scan_step_opts_t *opts, kda_stream_t stream) {
    kda_scan_step_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    kda_status_t st = check_scan(D, N, G, dtype);
    if (st != KDA_OK) return st;
    const int states = op.num_states ? op.num_states : requests;
    if (requests < 0 || requests > 65535 || op.num_states < 0 || (!op.state_indices && states < requests))
        return KDA_ERR_SHAPE;
    if (!A || (requests > 0 && (!u || !delta || !Bm || !Cm || !state || !y))) return KDA_ERR_NULL;
    if (!stride_ok(op.u_stride, D) || !stride_ok(op.delta_stride, D) || !stride_ok(op.z_stride, D) ||
        !stride_ok(op.y_stride, D) || !stride_ok(op.B_stride, (long long)G * N) ||
        !stride_ok(op.C_stride, (long long)G * N))
        return KDA_ERR_SHAPE;
    const int es = kda::esize(dtype);
    const void *ae[] = {u, delta, op.z, Bm, Cm, y}, *a4[] = {A, op.skip, op.delta_bias, op.state_indices};
    const void *a16[] = {state};
    if (misaligned(ae, es) || misaligned(a4, 4) || misaligned(a16, 16)) return KDA_ERR_ALIGN;
    const size_t ds = (size_t)D * 4;
    const Range in[] = {{u, requests, D, op.u_stride, es}, {delta, requests, D, op.delta_stride, es},
                        {op.z, op.z ? requests : 0, D, op.z_stride, es},
                        {Bm, requests, G * N, op.B_stride, es}, {Cm, requests, G * N, op.C_stride, es},
                        {A, (size_t)D * N * 4}, {op.skip, ds}, {op.delta_bias, ds},
                        {op.state_indices, (size_t)requests * 4}};
    const Range out[] = {{y, requests, D, op.y_stride, es}, {state, (size_t)states * D * N * 4}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (requests == 0) return KDA_OK;
    kda::ScanArgs a = {};
    a.u = u; a.delta = delta; a.z = op.z; a.B = Bm; a.C = Cm;
    a.A = A; a.skip = op.skip; a.delta_bias = op.delta_bias;
    a.y = y;
    a.D = D; a.N = N; a.G = G; a.dtype = dtype;
    a.softplus = !op.plain_delta;
    a.u_stride = op.u_stride; a.delta_stride = op.delta_stride; a.z_stride = op.z_stride;
    a.B_stride = op.B_stride; a.C_stride = op.C_stride; a.y_stride = op.y_stride;
    a.state = state;
    a.state_indices = op.state_indices;
    a.requests = requests;
    a.num_states = states;
    a.dbg = kda::debug_flags();
    return finish(kda::launch_scan_step(a, (cudaStream_t)stream));
}

// x's and the weight's copies where their rows are on no 16-byte boundary, and the partial sums.
size_t kda_linear_fwd_workspace_bytes(int M, int K, int N, int copies) {
    if (check_linear(M, K, N, KDA_BF16, 0) != KDA_OK || M == 0) return 0;
    return (copies & KDA_COPY_X ? copy_bytes(M, K) : 0) + (copies & KDA_COPY_WEIGHT ? copy_bytes(N, K) : 0) +
           (kda::small_gemm_ok(M, K) ? 0 : up256(kda::gemm_partial_bytes(M, N, K)));
}

int kda_linear_copies(const void *x, long long x_stride, const void *weight, long long weight_stride,
                      const void *dy, long long dy_stride) {
    return (rows_ok(x, x_stride) ? 0 : KDA_COPY_X) | (rows_ok(weight, weight_stride) ? 0 : KDA_COPY_WEIGHT) |
           (rows_ok(dy, dy_stride) ? 0 : KDA_COPY_DY);
}

kda_status_t kda_linear_fwd(const void *x, const void *weight, void *y, int M, int K, int N, int dtype,
                            const kda_linear_fwd_opts_t *opts, kda_stream_t stream) {
    kda_linear_fwd_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    kda_status_t st = check_linear(M, K, N, dtype, op.activation);
    if (st != KDA_OK) return st;
    if (!weight || (M > 0 && (!x || !y))) return KDA_ERR_NULL;
    if (!stride_ok(op.x_stride, K) || !stride_ok(op.weight_stride, K) || !stride_ok(op.y_stride, N) ||
        !stride_ok(op.residual_stride, N))
        return KDA_ERR_SHAPE;
    const void *a2[] = {x, weight, y, op.bias, op.residual, op.saved}, *a256[] = {op.workspace};
    if (misaligned(a2, 2) || misaligned(a256, 256)) return KDA_ERR_ALIGN;
    const int copies = kda_linear_copies(x, op.x_stride, weight, op.weight_stride, nullptr, 0);
    const size_t need = kda_linear_fwd_workspace_bytes(M, K, N, copies);
    if (need && (!op.workspace || op.workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const Range in[] = {{x, M, K, op.x_stride, 2}, {weight, N, K, op.weight_stride, 2},
                        {op.bias, (size_t)N * 2}, {op.residual, op.residual ? M : 0, N, op.residual_stride, 2}};
    const Range out[] = {{y, M, N, op.y_stride, 2}, {op.saved, (size_t)M * N * 2},
                         {need ? op.workspace : nullptr, need}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    if (M == 0) return KDA_OK;
    Work w = {(char *)op.workspace};
    Copies c;
    c.add(x, op.x_stride, M, K, w);
    c.add(weight, op.weight_stride, N, K, w);
    cudaError_t e = c.run((cudaStream_t)stream);
    if (e != cudaSuccess) return finish(e);
    kda::GemmArgs a = {};
    a.A = x; a.B = weight;
    a.lda = op.x_stride; a.ldb = op.weight_stride;
    a.M = M; a.N = N; a.K = K;
    a.bias = op.bias; a.residual = op.residual; a.y = y; a.pre = op.saved;
    a.ldr = op.residual_stride; a.ldy = op.y_stride; a.ldp = N;
    a.act = op.activation;
    a.fp16 = dtype == KDA_FP16;
    a.partial = (float *)w.at;
    a.partial_floats = kda::gemm_partial_bytes(M, N, K) / 4;
    a.dbg = kda::debug_flags();
    a.give_up = kda::debug_give_up();
    return finish(kda::small_gemm_ok(M, K) ? kda::launch_small_gemm(a, (cudaStream_t)stream)
                                        : kda::launch_gemm(a, (cudaStream_t)stream));
}

// dpre, its column sums, x's and the weight's copies, the partial sums (one product after the other)
size_t kda_linear_bwd_workspace_bytes(int M, int K, int N, int activation, int copies, int wanted) {
    if (check_linear(M, K, N, KDA_BF16, activation) != KDA_OK || M == 0) return 0;
    size_t s = 0;
    if (activation != KDA_ACT_NONE || (copies & KDA_COPY_DY)) s += copy_bytes(M, N);
    if (wanted & KDA_GRAD_BIAS) s += up256((size_t)kda::dact_partials(M, N) * N * 4);
    if ((wanted & KDA_GRAD_WEIGHT) && (copies & KDA_COPY_X)) s += copy_bytes(M, K);
    if ((wanted & KDA_GRAD_X) && (copies & KDA_COPY_WEIGHT)) s += copy_bytes(N, K);
    size_t p = 0, q;
    if (wanted & KDA_GRAD_X) p = kda::gemm_partial_bytes(M, K, N);
    if ((wanted & KDA_GRAD_WEIGHT) && (q = kda::gemm_partial_bytes(N, K, M)) > p) p = q;
    return s + up256(p);
}

kda_status_t kda_linear_bwd(const void *dy, const void *x, const void *weight, void *dx, void *dweight,
                            void *dbias, int M, int K, int N, int dtype, const kda_linear_bwd_opts_t *opts,
                            kda_stream_t stream) {
    kda_linear_bwd_opts_t op;
    memset(&op, 0, sizeof(op));
    if (opts) op = *opts;
    kda_status_t st = check_linear(M, K, N, dtype, op.activation);
    if (st != KDA_OK) return st;
    if (M > 0 && (!dy || (dweight && !x) || (dx && !weight) || (op.activation != KDA_ACT_NONE && !op.saved)))
        return KDA_ERR_NULL;
    if (!stride_ok(op.x_stride, K) || !stride_ok(op.weight_stride, K) || !stride_ok(op.dy_stride, N) ||
        !stride_ok(op.dx_stride, K))
        return KDA_ERR_SHAPE;
    const void *a2[] = {dy, x, weight, dx, dweight, dbias, op.saved}, *a256[] = {op.workspace};
    if (misaligned(a2, 2) || misaligned(a256, 256)) return KDA_ERR_ALIGN;
    const int copies = kda_linear_copies(x, op.x_stride, weight, op.weight_stride, dy, op.dy_stride);
    const int wanted = (dx ? KDA_GRAD_X : 0) | (dweight ? KDA_GRAD_WEIGHT : 0) | (dbias ? KDA_GRAD_BIAS : 0);
    const size_t need = kda_linear_bwd_workspace_bytes(M, K, N, op.activation, copies, wanted);
    if (need && (!op.workspace || op.workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const bool act = op.activation != KDA_ACT_NONE;
    const Range in[] = {{dy, M, N, op.dy_stride, 2}, {x, x ? M : 0, K, op.x_stride, 2},
                        {weight, weight ? N : 0, K, op.weight_stride, 2},
                        {act ? op.saved : nullptr, (size_t)M * N * 2}};
    const Range out[] = {{dx, dx ? M : 0, K, op.dx_stride, 2}, {dweight, (size_t)N * K * 2},
                         {dbias, (size_t)N * 2}, {need ? op.workspace : nullptr, need}};
    if (overlap(out, in)) return KDA_ERR_OVERLAP;
    if ((st = kda::require_device()) != KDA_OK) return st;
    (void)cudaGetLastError();
    const cudaStream_t cs = (cudaStream_t)stream;
    if (M == 0) {  // sums of nothing
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)N * K * 2, cs);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)N * 2, cs);
        return finish(e);
    }
    Work w = {(char *)op.workspace};
    const void *g = dy;
    long long ldg = op.dy_stride;
    if (act || dbias || (copies & KDA_COPY_DY)) {
        kda::DActArgs d = {};
        d.dy = dy; d.lddy = op.dy_stride;
        d.pre = op.saved; d.ldp = N;
        if (act || (copies & KDA_COPY_DY)) {
            ldg = up8(N);
            d.dpre = w.take((size_t)M * ldg * 2);
            d.ldd = ldg;
            g = d.dpre;
        }
        if (dbias) {
            d.dbias = dbias;
            d.partial_floats = (size_t)kda::dact_partials(M, N) * N;
            d.partial = (float *)w.take(d.partial_floats * 4);
        }
        d.M = M; d.N = N; d.act = op.activation; d.fp16 = dtype == KDA_FP16;
        d.dbg = kda::debug_flags();
        const cudaError_t e = kda::launch_dact(d, cs);
        if (e != cudaSuccess) return finish(e);
    }
    kda::GemmArgs a = {};
    a.fp16 = dtype == KDA_FP16;
    a.dbg = kda::debug_flags();
    a.give_up = kda::debug_give_up();
    Copies c;
    if (dweight) c.add(x, op.x_stride, M, K, w);
    if (dx) c.add(weight, op.weight_stride, N, K, w);
    cudaError_t e = c.run(cs);
    if (e != cudaSuccess) return finish(e);
    a.partial = (float *)w.at;
    if (dx) {  // dpre weight: contracted over the weight's rows
        a.A = g; a.lda = ldg;
        a.B = weight; a.ldb = op.weight_stride; a.b_mn = true;
        a.M = M; a.N = K; a.K = N;
        a.partial_floats = kda::gemm_partial_bytes(M, K, N) / 4;
        a.y = dx; a.ldy = op.dx_stride;
        if ((e = kda::launch_gemm(a, cs)) != cudaSuccess) return finish(e);
    }
    if (dweight) {  // dpre^T x: contracted over the rows of both
        a.A = g; a.lda = ldg; a.a_mn = true;
        a.B = x; a.ldb = op.x_stride; a.b_mn = true;
        a.M = N; a.N = K; a.K = M;
        a.partial_floats = kda::gemm_partial_bytes(N, K, M) / 4;
        a.y = dweight; a.ldy = K;
        if ((e = kda::launch_gemm(a, cs)) != cudaSuccess) return finish(e);
    }
    return KDA_OK;
}

}  // extern "C"
