// The short way from Python to every entry point but the intra-chunk ones: checks
// of the arguments, outputs and the call in one C++ function each.  Small calls are bound by
// what the host does between two launches: a step for one request took 15 us of Python around
// a kernel of 2.4 us.
//
// Every function returns None for arguments that it does not take as they are, and when the
// library refuses the call.  The Python functions then go their own way, which takes everything
// that is allowed and says what is wrong with the rest; nothing is accepted here that they would
// refuse.  The first arguments are the addresses of the library's functions, so that calls can
// be sent through another build of it.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kda.h"

namespace {

constexpr int64_t K = 128;

using at::ScalarType;
using at::Tensor;

const Tensor *tensor(PyObject *o) {
    return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// An optional argument: false if it is neither None nor a tensor.
bool optional(PyObject *o, const Tensor *&t) {
    t = o == Py_None ? nullptr : tensor(o);
    return t || o == Py_None;
}

bool fits(const Tensor *t, at::IntArrayRef shape, ScalarType type, int dev) {
    return t && t->scalar_type() == type && t->layout() == at::kStrided && t->is_cuda() &&
           t->get_device() == dev && t->sizes() == shape && t->is_contiguous();
}

// 0 (the library's default) for None; a scale of 0 is left to the checks in Python.
bool scale_of(PyObject *o, float &scale) {
    scale = 0.f;
    if (o == Py_None) return true;
    if (!PyFloat_Check(o)) return false;
    scale = (float)PyFloat_AS_DOUBLE(o);
    return scale != 0.f;
}

template <class F> F function(PyObject *address) { return (F)PyLong_AsVoidPtr(address); }

int type_of(ScalarType t) {
    return t == at::kBFloat16 ? KDA_BF16 : t == at::kHalf ? KDA_FP16 : t == at::kFloat ? KDA_FP32 : -1;
}

Tensor empty(at::IntArrayRef shape, ScalarType type, const Tensor &like) {
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
Tensor bytes(size_t n, const Tensor &like) { return empty({(int64_t)n}, at::kByte, like); }

PyObject *wrap(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <size_t N> PyObject *wrap_all(const Tensor (&ts)[N]) {
    PyObject *out = PyTuple_New(N);
    if (!out) return nullptr;
    for (size_t i = 0; i < N; ++i) {
        PyObject *o = wrap(ts[i]);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, o);
    }
    return out;
}

// q, k, v, gate, beta with `lead` leading dimensions.
struct Inputs {
    const Tensor *q, *k, *v, *gate, *beta;
    ScalarType type;
    int dev, H, HV, dtype;

    bool read(PyObject *const *o, size_t lead) {
        q = tensor(o[0]); k = tensor(o[1]); v = tensor(o[2]); gate = tensor(o[3]);
        beta = tensor(o[4]);
        if (!q || !k || !v || !gate || !beta || !q->is_cuda()) return false;
        type = q->scalar_type();
        if (type != at::kBFloat16 && type != at::kHalf) return false;
        dtype = type_of(type);
        const at::IntArrayRef s = q->sizes(), vs = v->sizes();
        if (s.size() != lead + 2 || vs.size() != lead + 2) return false;
        for (int64_t n : s)
            if (n > INT_MAX) return false;
        dev = q->get_device();
        if (s[lead + 1] != K || s[lead] == 0 || vs[lead] > INT_MAX || vs[lead] % s[lead] ||
            vs[lead + 1] != K || vs.slice(0, lead) != s.slice(0, lead))
            return false;
        H = (int)s[lead];
        HV = (int)vs[lead];
        return fits(q, s, type, dev) && fits(k, s, type, dev) && fits(v, vs, type, dev) &&
               fits(gate, vs, at::kFloat, dev) && fits(beta, vs.slice(0, lead + 1), at::kFloat, dev) &&
               c10::cuda::current_device() == dev;
    }
};

kda_stream_t stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

// A call into the library without Python's lock: a launch may wait for a full queue.
template <class F> bool call(const F &f) {
    kda_status_t rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc == KDA_OK;
}

// (kda_step, q, k, v, gate, beta, state, scale, state_indices, o)
PyObject *step(PyObject *const *a) {
    Inputs x;
    const Tensor *state = tensor(a[6]), *index, *given;
    kda_step_opts_t op = {};
    if (!x.read(a + 1, 1) || !state || state->dim() != 4 || !scale_of(a[7], op.scale) ||
        !optional(a[8], index) || !optional(a[9], given))
        Py_RETURN_NONE;
    const int64_t N = x.q->size(0), states = state->size(0);
    if ((!index && states != N) || states > INT_MAX ||
        !fits(state, {states, x.HV, K, K}, at::kFloat, x.dev) ||
        (index && !fits(index, {N}, at::kInt, x.dev)) ||
        (given && !fits(given, x.v->sizes(), x.type, x.dev)))
        Py_RETURN_NONE;
    op.HV = x.HV;
    op.num_states = (int)states;
    if (index) op.state_indices = (const int *)index->data_ptr();
    const Tensor o = given ? *given : empty(x.v->sizes(), x.type, *x.v);
    const kda_stream_t stream = stream_of(x.dev);
    if (!call([&] {
            return function<decltype(&kda_step)>(a[0])(
                x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), (const float *)x.gate->data_ptr(),
                (const float *)x.beta->data_ptr(), (float *)state->data_ptr(), o.data_ptr(), (int)N,
                x.H, (kda_dtype_t)x.dtype, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap(o);
}

// (kda_chunk_fwd, kda_chunk_saved_bytes, q, k, v, gate, beta, scale, initial_state,
//  output_final_state, save): sequences of one length
PyObject *chunk_fwd(PyObject *const *a) {
    Inputs x;
    const Tensor *initial;
    kda_chunk_fwd_opts_t op = {};
    if (!x.read(a + 2, 2) || !scale_of(a[7], op.scale) || !optional(a[8], initial))
        Py_RETURN_NONE;
    const int64_t B = x.q->size(0), T = x.q->size(1);
    const int want_final = PyObject_IsTrue(a[9]), save = PyObject_IsTrue(a[10]);
    if (want_final < 0 || save < 0) return nullptr;
    if (B == 0 || (initial && !fits(initial, {B, x.HV, K, K}, at::kFloat, x.dev))) Py_RETURN_NONE;
    op.HV = x.HV;
    if (initial) op.initial_state = (const float *)initial->data_ptr();
    Tensor out[3] = {empty(x.v->sizes(), x.type, *x.v)};
    if (want_final) {
        out[1] = empty({B, x.HV, K, K}, at::kFloat, *x.q);
        op.final_state = (float *)out[1].data_ptr();
    }
    if (save) {
        op.saved_bytes = function<decltype(&kda_chunk_saved_bytes)>(a[1])(
            (int)B, (int)T, x.HV, 0, (kda_dtype_t)x.dtype, initial || want_final);
        out[2] = bytes(op.saved_bytes, *x.q);
        op.saved = out[2].data_ptr();
    }
    const kda_stream_t stream = stream_of(x.dev);
    if (!call([&] {
            return function<decltype(&kda_chunk_fwd)>(a[0])(
                x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), (const float *)x.gate->data_ptr(),
                (const float *)x.beta->data_ptr(), out[0].data_ptr(), (int)B, (int)T, x.H,
                (kda_dtype_t)x.dtype, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// (kda_chunk_bwd, kda_chunk_saved_bytes, kda_chunk_bwd_workspace_bytes, q, k, v, gate, beta, do,
//  saved, scale): sequences of one length, no gradient of a state
PyObject *chunk_bwd(PyObject *const *a) {
    Inputs x;
    const Tensor *dout = tensor(a[8]), *saved = tensor(a[9]);
    kda_chunk_bwd_opts_t op = {};
    if (!x.read(a + 3, 2) || !dout || !saved || !scale_of(a[10], op.scale)) Py_RETURN_NONE;
    const int64_t B = x.q->size(0), T = x.q->size(1), n = saved->numel();
    if (B == 0 || !fits(dout, x.v->sizes(), x.type, x.dev) || !fits(saved, {n}, at::kByte, x.dev))
        Py_RETURN_NONE;
    const auto dtype = (kda_dtype_t)x.dtype;
    const auto saved_bytes = function<decltype(&kda_chunk_saved_bytes)>(a[1]);
    if ((size_t)n != saved_bytes((int)B, (int)T, x.HV, 0, dtype, 0) &&
        (size_t)n != saved_bytes((int)B, (int)T, x.HV, 0, dtype, 1))
        Py_RETURN_NONE;
    op.HV = x.HV;
    op.saved = saved->data_ptr();
    op.saved_bytes = (size_t)n;
    op.workspace_bytes = function<decltype(&kda_chunk_bwd_workspace_bytes)>(a[2])(
        (int)B, (int)T, x.H, x.HV, 0, dtype, op.saved_bytes);
    const Tensor work = bytes(op.workspace_bytes, *x.q);
    op.workspace = work.data_ptr();
    const Tensor out[6] = {empty(x.q->sizes(), x.type, *x.q), empty(x.q->sizes(), x.type, *x.q),
                           empty(x.v->sizes(), x.type, *x.q), empty(x.v->sizes(), x.type, *x.q),
                           empty(x.beta->sizes(), x.type, *x.q)};
    const kda_stream_t stream = stream_of(x.dev);
    if (!call([&] {
            return function<decltype(&kda_chunk_bwd)>(a[0])(
                x.q->data_ptr(), x.k->data_ptr(), (const float *)x.gate->data_ptr(),
                (const float *)x.beta->data_ptr(), dout->data_ptr(), out[0].data_ptr(),
                out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(), (int)B,
                (int)T, x.H, dtype, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// x and the parameters of a layer norm; everything contiguous.
struct Norm {
    const Tensor *x, *weight, *bias;
    int dev, width, dtype, wdtype;
    int64_t rows;

    bool read(PyObject *ox, PyObject *ow, PyObject *ob) {
        x = tensor(ox);
        if (!x || !optional(ow, weight) || !optional(ob, bias) || !x->is_cuda() || x->dim() == 0 ||
            x->size(-1) == 0 || x->size(-1) > INT_MAX || type_of(x->scalar_type()) < 0)
            return false;
        dev = x->get_device();
        width = (int)x->size(-1);
        rows = x->numel() / width;
        const ScalarType wt = weight ? weight->scalar_type()
                              : bias ? bias->scalar_type()
                                     : x->scalar_type();
        dtype = type_of(x->scalar_type());
        wdtype = type_of(wt);
        return (wt == x->scalar_type() || wt == at::kFloat) && like_x(x) &&
               (!weight || fits(weight, {width}, wt, dev)) && (!bias || fits(bias, {width}, wt, dev)) &&
               c10::cuda::current_device() == dev;
    }
    bool like_x(const Tensor *t) const { return fits(t, x->sizes(), x->scalar_type(), dev); }
    const void *w() const { return weight ? weight->data_ptr() : nullptr; }
};

// (kda_layer_norm_fwd, x, weight, bias, eps)
PyObject *layer_norm_fwd(PyObject *const *a) {
    Norm n;
    if (!PyFloat_Check(a[4]) || !n.read(a[1], a[2], a[3])) Py_RETURN_NONE;
    const Tensor out[3] = {empty(n.x->sizes(), n.x->scalar_type(), *n.x),
                           empty({n.rows}, at::kFloat, *n.x), empty({n.rows}, at::kFloat, *n.x)};
    const float eps = (float)PyFloat_AS_DOUBLE(a[4]);
    const kda_stream_t stream = stream_of(n.dev);
    if (!call([&] {
            return function<decltype(&kda_layer_norm_fwd)>(a[0])(
                n.x->data_ptr(), n.w(), n.bias ? n.bias->data_ptr() : nullptr, out[0].data_ptr(),
                (float *)out[1].data_ptr(), (float *)out[2].data_ptr(), n.rows, n.width, eps,
                n.dtype, n.wdtype, n.width, n.width, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// (kda_layer_norm_bwd, kda_layer_norm_bwd_workspace_bytes, dy, x, weight, mean, rstd)
PyObject *layer_norm_bwd(PyObject *const *a) {
    Norm n;
    const Tensor *dy = tensor(a[2]), *mean = tensor(a[5]), *rstd = tensor(a[6]);
    if (!n.read(a[3], a[4], Py_None) || !n.like_x(dy) || !fits(mean, {n.rows}, at::kFloat, n.dev) ||
        !fits(rstd, {n.rows}, at::kFloat, n.dev))
        Py_RETURN_NONE;
    const Tensor out[3] = {empty(n.x->sizes(), n.x->scalar_type(), *n.x),
                           empty({n.width}, at::kFloat, *n.x), empty({n.width}, at::kFloat, *n.x)};
    const size_t need =
        function<decltype(&kda_layer_norm_bwd_workspace_bytes)>(a[1])(n.rows, n.width);
    const Tensor work = bytes(need, *n.x);
    const kda_stream_t stream = stream_of(n.dev);
    if (!call([&] {
            return function<decltype(&kda_layer_norm_bwd)>(a[0])(
                dy->data_ptr(), n.x->data_ptr(), n.w(), (const float *)mean->data_ptr(),
                (const float *)rstd->data_ptr(), out[0].data_ptr(), (float *)out[1].data_ptr(),
                (float *)out[2].data_ptr(), n.rows, n.width, n.dtype, n.wdtype, n.width, n.width,
                n.width, work.data_ptr(), need, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// Elements between the rows of a tensor whose last `tail` dimensions are one contiguous row and whose
// leading ones are one evenly spaced run of rows; false for any other.
bool row_stride(const Tensor *t, at::IntArrayRef shape, ScalarType type, int dev, size_t tail,
                long long &stride) {
    if (!t || t->scalar_type() != type || t->layout() != at::kStrided || !t->is_cuda() ||
        t->get_device() != dev || t->sizes() != shape)
        return false;
    const at::IntArrayRef st = t->strides();
    int64_t width = 1;
    const size_t lead = shape.size() - tail;
    for (size_t i = shape.size(); i-- > lead;) {
        if (shape[i] > 1 && st[i] != width) return false;
        width *= shape[i];
    }
    int64_t step = width, run = 0;
    bool any = false;
    for (size_t i = lead; i-- > 0;) {
        if (shape[i] == 1) continue;
        if (!any)
            step = st[i];
        else if (st[i] != run)
            return false;
        any = true;
        run = shape[i] * st[i];
    }
    if (t->numel() == 0) step = width;
    if (step < width) return false;  // rows on one another: an expanded dimension
    stride = step;
    return true;
}
// Sequences packed along T, 0 without cu_seqlens; -1 for a table that is not taken.
int sequences(PyObject *o, int64_t B, int dev, const Tensor *&cu) {
    if (!optional(o, cu)) return -1;
    if (!cu) return 0;
    const int64_t n = cu->numel();
    return B == 1 && n >= 2 && n <= INT_MAX && fits(cu, {n}, at::kInt, dev) ? (int)n - 1 : -1;
}
const void *address(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
bool within(at::IntArrayRef s) {
    for (int64_t n : s)
        if (n > INT_MAX) return false;
    return true;
}

// x and the parameters of a convolution.
struct Conv {
    const Tensor *x, *weight, *bias;
    ScalarType type;
    int dev, D, W, dtype, wdtype;
    long long stride;

    bool read(PyObject *ox, PyObject *ow, PyObject *ob, int64_t lead) {
        x = tensor(ox);
        weight = tensor(ow);
        if (!x || !weight || !optional(ob, bias) || !x->is_cuda() || x->dim() != lead + 1 ||
            weight->dim() != 2 || !within(x->sizes()) || type_of(x->scalar_type()) < 0)
            return false;
        type = x->scalar_type();
        dev = x->get_device();
        D = (int)x->size(lead);
        W = (int)weight->size(1);
        const ScalarType wt = weight->scalar_type();
        dtype = type_of(type);
        wdtype = type_of(wt);
        return D > 0 && W >= 2 && W <= 4 && (wt == type || wt == at::kFloat) &&
               row_stride(x, x->sizes(), type, dev, 1, stride) && fits(weight, {D, W}, wt, dev) &&
               (!bias || fits(bias, {D}, wt, dev)) && c10::cuda::current_device() == dev;
    }
};

// (kda_conv_fwd, x, weight, bias, initial_state, silu, output_final_state, cu_seqlens)
PyObject *conv_fwd(PyObject *const *a) {
    Conv c;
    const Tensor *initial, *cu;
    if (!c.read(a[1], a[2], a[3], 2) || !optional(a[4], initial)) Py_RETURN_NONE;
    const int64_t B = c.x->size(0), T = c.x->size(1);
    const int silu = PyObject_IsTrue(a[5]), want = PyObject_IsTrue(a[6]), seqs = sequences(a[7], B, c.dev, cu);
    if (silu < 0 || want < 0) return nullptr;
    const int64_t n = cu ? seqs : B;
    if (seqs < 0 || B == 0 || (initial && !fits(initial, {n, c.W - 1, c.D}, c.type, c.dev))) Py_RETURN_NONE;
    Tensor out[2] = {empty(c.x->sizes(), c.type, *c.x)};
    if (want) out[1] = empty({n, c.W - 1, c.D}, c.type, *c.x);
    kda_conv_fwd_opts_t op = {};
    op.initial_state = address(initial);
    op.final_state = want ? out[1].data_ptr() : nullptr;
    op.cu_seqlens = (const int *)address(cu);
    op.num_seqs = seqs;
    op.zero_rest = 1;
    op.x_stride = c.stride;
    const kda_stream_t stream = stream_of(c.dev);
    if (!call([&] {
            return function<decltype(&kda_conv_fwd)>(a[0])(
                c.x->data_ptr(), c.weight->data_ptr(), address(c.bias), out[0].data_ptr(), (int)B, (int)T,
                c.D, c.W, c.dtype, c.wdtype, silu ? KDA_ACT_SILU : KDA_ACT_NONE, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// (kda_conv_bwd, kda_conv_bwd_workspace_bytes, dy, x, weight, bias, silu, cu_seqlens): no states
PyObject *conv_bwd(PyObject *const *a) {
    Conv c;
    const Tensor *dy = tensor(a[2]), *cu;
    kda_conv_bwd_opts_t op = {};
    if (!c.read(a[3], a[4], a[5], 2) || !row_stride(dy, c.x->sizes(), c.type, c.dev, 1, op.dy_stride))
        Py_RETURN_NONE;
    const int64_t B = c.x->size(0), T = c.x->size(1);
    const int silu = PyObject_IsTrue(a[6]), seqs = sequences(a[7], B, c.dev, cu);
    if (silu < 0) return nullptr;
    if (seqs < 0 || B == 0) Py_RETURN_NONE;
    const Tensor out[4] = {empty(c.x->sizes(), c.type, *c.x), empty({c.D, c.W}, at::kFloat, *c.x),
                           empty({c.D}, at::kFloat, *c.x)};
    op.workspace_bytes = function<decltype(&kda_conv_bwd_workspace_bytes)>(a[1])((int)B, (int)T, c.D, c.W, seqs);
    const Tensor work = bytes(op.workspace_bytes, *c.x);
    op.workspace = work.data_ptr();
    op.cu_seqlens = (const int *)address(cu);
    op.num_seqs = seqs;
    op.zero_rest = 1;
    op.x_stride = c.stride;
    const kda_stream_t stream = stream_of(c.dev);
    if (!call([&] {
            return function<decltype(&kda_conv_bwd)>(a[0])(
                dy->data_ptr(), c.x->data_ptr(), c.weight->data_ptr(), address(c.bias), out[0].data_ptr(),
                (float *)out[1].data_ptr(), (float *)out[2].data_ptr(), (int)B, (int)T, c.D, c.W, c.dtype,
                c.wdtype, silu ? KDA_ACT_SILU : KDA_ACT_NONE, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// (kda_conv_step, x, state, weight, bias, silu, state_indices)
PyObject *conv_step(PyObject *const *a) {
    Conv c;
    const Tensor *state = tensor(a[2]), *index;
    const int silu = PyObject_IsTrue(a[5]);
    if (silu < 0) return nullptr;
    if (!c.read(a[1], a[3], a[4], 1) || !state || state->dim() != 3 || !optional(a[6], index)) Py_RETURN_NONE;
    const int64_t N = c.x->size(0), states = state->size(0);
    if ((!index && states != N) || states > INT_MAX || !fits(state, {states, c.W - 1, c.D}, c.type, c.dev) ||
        (index && !fits(index, {N}, at::kInt, c.dev)))
        Py_RETURN_NONE;
    const Tensor y = empty(c.x->sizes(), c.type, *c.x);
    kda_conv_step_opts_t op = {};
    op.state_indices = (const int *)address(index);
    op.num_states = (int)states;
    op.x_stride = c.stride;
    const kda_stream_t stream = stream_of(c.dev);
    if (!call([&] {
            return function<decltype(&kda_conv_step)>(a[0])(
                c.x->data_ptr(), c.weight->data_ptr(), address(c.bias), state->data_ptr(), y.data_ptr(), (int)N,
                c.D, c.W, c.dtype, c.wdtype, silu ? KDA_ACT_SILU : KDA_ACT_NONE, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap(y);
}

// The inputs of a scan: u, delta, A, B, C, and D, z, delta_bias.
struct Scan {
    const Tensor *u, *delta, *A, *B, *C, *skip, *z, *bias;
    ScalarType type;
    int dev, D, N, G, dtype;
    long long su, sd, sz = 0, sB, sC;

    bool read(PyObject *const *o, PyObject *const *more, size_t lead) {
        u = tensor(o[0]); delta = tensor(o[1]); A = tensor(o[2]); B = tensor(o[3]); C = tensor(o[4]);
        if (!u || !delta || !A || !B || !C || !optional(more[0], skip) || !optional(more[1], z) ||
            !optional(more[2], bias) || !u->is_cuda() || u->dim() != (int64_t)lead + 1 || A->dim() != 2 ||
            B->dim() != (int64_t)lead + 2 || type_of(u->scalar_type()) < 0)
            return false;
        type = u->scalar_type();
        dtype = type_of(type);
        dev = u->get_device();
        const at::IntArrayRef s = u->sizes(), v = B->sizes();
        if (!within(s) || !within(v) || A->size(1) < 1 || A->size(1) > 64 || v[lead] < 1 || s[lead] < 1 ||
            s[lead] % v[lead] || v[lead + 1] != A->size(1) || v.slice(0, lead) != s.slice(0, lead))
            return false;
        D = (int)s[lead];
        N = (int)A->size(1);
        G = (int)v[lead];
        return fits(A, {D, N}, at::kFloat, dev) && row_stride(u, s, type, dev, 1, su) &&
               row_stride(delta, s, type, dev, 1, sd) && row_stride(B, v, type, dev, 2, sB) &&
               row_stride(C, v, type, dev, 2, sC) && (!z || row_stride(z, s, type, dev, 1, sz)) &&
               (!skip || fits(skip, {D}, at::kFloat, dev)) && (!bias || fits(bias, {D}, at::kFloat, dev)) &&
               c10::cuda::current_device() == dev;
    }
    template <class Op> void options(Op &op) const {
        op.skip = (const float *)address(skip);
        op.delta_bias = (const float *)address(bias);
        op.z = address(z);
        op.u_stride = su; op.delta_stride = sd; op.z_stride = sz; op.B_stride = sB; op.C_stride = sC;
    }
};

// (kda_scan_fwd, kda_scan_saved_bytes, kda_scan_fwd_workspace_bytes, u, delta, A, B, C, D, z,
//  delta_bias, initial_state, output_final_state, save, cu_seqlens)
PyObject *scan_fwd(PyObject *const *a) {
    Scan x;
    const Tensor *initial, *cu;
    kda_scan_fwd_opts_t op = {};
    if (!x.read(a + 3, a + 8, 2) || !optional(a[11], initial)) Py_RETURN_NONE;
    const int64_t B = x.u->size(0), T = x.u->size(1);
    const int want = PyObject_IsTrue(a[12]), save = PyObject_IsTrue(a[13]), seqs = sequences(a[14], B, x.dev, cu);
    if (want < 0 || save < 0) return nullptr;
    const int64_t n = cu ? seqs : B;
    if (seqs < 0 || B == 0 || (initial && !fits(initial, {n, x.D, x.N}, at::kFloat, x.dev))) Py_RETURN_NONE;
    x.options(op);
    op.initial_state = (const float *)address(initial);
    op.cu_seqlens = (const int *)address(cu);
    op.num_seqs = seqs;
    op.zero_rest = 1;
    Tensor out[3] = {empty(x.u->sizes(), x.type, *x.u)};
    if (want) {
        out[1] = empty({n, x.D, x.N}, at::kFloat, *x.u);
        op.final_state = (float *)out[1].data_ptr();
    }
    if (save) {
        op.saved_bytes = function<decltype(&kda_scan_saved_bytes)>(a[1])((int)B, (int)T, x.D, x.N, seqs);
        out[2] = bytes(op.saved_bytes, *x.u);
        op.saved = out[2].data_ptr();
    }
    op.workspace_bytes =
        function<decltype(&kda_scan_fwd_workspace_bytes)>(a[2])((int)B, (int)T, x.D, x.N, x.G, seqs);
    Tensor work;
    if (op.workspace_bytes) {
        work = bytes(op.workspace_bytes, *x.u);
        op.workspace = work.data_ptr();
    }
    const kda_stream_t stream = stream_of(x.dev);
    if (!call([&] {
            return function<decltype(&kda_scan_fwd)>(a[0])(
                x.u->data_ptr(), x.delta->data_ptr(), (const float *)x.A->data_ptr(), x.B->data_ptr(),
                x.C->data_ptr(), out[0].data_ptr(), (int)B, (int)T, x.D, x.N, x.G, x.dtype, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// (kda_scan_bwd, kda_scan_saved_bytes, kda_scan_bwd_workspace_bytes, dy, u, delta, A, B, C, saved, D,
//  z, delta_bias, cu_seqlens): no states
PyObject *scan_bwd(PyObject *const *a) {
    Scan x;
    const Tensor *dy = tensor(a[3]), *saved = tensor(a[9]), *cu;
    kda_scan_bwd_opts_t op = {};
    if (!saved || !x.read(a + 4, a + 10, 2) || !row_stride(dy, x.u->sizes(), x.type, x.dev, 1, op.dy_stride))
        Py_RETURN_NONE;
    const int64_t B = x.u->size(0), T = x.u->size(1), n = saved->numel();
    const int seqs = sequences(a[13], B, x.dev, cu);
    if (seqs < 0 || B == 0 || !fits(saved, {n}, at::kByte, x.dev) ||
        (size_t)n != function<decltype(&kda_scan_saved_bytes)>(a[1])((int)B, (int)T, x.D, x.N, seqs))
        Py_RETURN_NONE;
    const at::IntArrayRef s = x.u->sizes(), v = x.B->sizes();
    Tensor out[9] = {empty(s, x.type, *x.u), empty(s, x.type, *x.u), empty({x.D, x.N}, at::kFloat, *x.u),
                     empty(v, x.type, *x.u), empty(v, x.type, *x.u)};
    x.options(op);
    if (x.skip) {
        out[5] = empty({x.D}, at::kFloat, *x.u);
        op.dskip = (float *)out[5].data_ptr();
    }
    if (x.z) {
        out[6] = empty(s, x.type, *x.u);
        op.dz = out[6].data_ptr();
    }
    if (x.bias) {
        out[7] = empty({x.D}, at::kFloat, *x.u);
        op.ddelta_bias = (float *)out[7].data_ptr();
    }
    op.saved = saved->data_ptr();
    op.saved_bytes = (size_t)n;
    op.cu_seqlens = (const int *)address(cu);
    op.num_seqs = seqs;
    op.zero_rest = 1;
    op.workspace_bytes =
        function<decltype(&kda_scan_bwd_workspace_bytes)>(a[2])((int)B, (int)T, x.D, x.N, x.G, seqs);
    const Tensor work = bytes(op.workspace_bytes, *x.u);
    op.workspace = work.data_ptr();
    const kda_stream_t stream = stream_of(x.dev);
    if (!call([&] {
            return function<decltype(&kda_scan_bwd)>(a[0])(
                dy->data_ptr(), x.u->data_ptr(), x.delta->data_ptr(), (const float *)x.A->data_ptr(),
                x.B->data_ptr(), x.C->data_ptr(), out[0].data_ptr(), out[1].data_ptr(),
                (float *)out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(), (int)B, (int)T, x.D, x.N, x.G,
                x.dtype, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// (kda_scan_step, u, delta, A, B, C, state, D, z, delta_bias, state_indices)
PyObject *scan_step(PyObject *const *a) {
    Scan x;
    const Tensor *state = tensor(a[6]), *index;
    kda_scan_step_opts_t op = {};
    if (!x.read(a + 1, a + 7, 1) || !state || state->dim() != 3 || !optional(a[10], index)) Py_RETURN_NONE;
    const int64_t N = x.u->size(0), states = state->size(0);
    if ((!index && states != N) || states > INT_MAX || !fits(state, {states, x.D, x.N}, at::kFloat, x.dev) ||
        (index && !fits(index, {N}, at::kInt, x.dev)))
        Py_RETURN_NONE;
    const Tensor y = empty(x.u->sizes(), x.type, *x.u);
    x.options(op);
    op.state_indices = (const int *)address(index);
    op.num_states = (int)states;
    const kda_stream_t stream = stream_of(x.dev);
    if (!call([&] {
            return function<decltype(&kda_scan_step)>(a[0])(
                x.u->data_ptr(), x.delta->data_ptr(), (const float *)x.A->data_ptr(), x.B->data_ptr(),
                x.C->data_ptr(), (float *)state->data_ptr(), y.data_ptr(), (int)N, x.D, x.N, x.G, x.dtype, &op,
                stream);
        }))
        Py_RETURN_NONE;
    return wrap(y);
}

// x [..., K] and weight [N, K] of a matrix product.
struct Linear {
    const Tensor *x, *weight;
    ScalarType type;
    int dev, M, K, N, dtype, act;
    long long sx, sw;
    c10::SmallVector<int64_t, 8> shape;  // of y

    bool read(PyObject *ox, PyObject *ow, PyObject *oa) {
        x = tensor(ox);
        weight = tensor(ow);
        if (!x || !weight || !PyLong_Check(oa) || !x->is_cuda() || x->dim() == 0 || weight->dim() != 2) return false;
        type = x->scalar_type();
        if (type != at::kBFloat16 && type != at::kHalf) return false;
        dtype = type_of(type);
        dev = x->get_device();
        act = (int)PyLong_AsLong(oa);
        const int64_t k = x->size(-1), n = weight->size(0), m = k ? x->numel() / k : 0;
        if (k < 1 || n < 1 || k > INT_MAX || n > INT_MAX || m > INT_MAX || weight->size(1) != k) return false;
        M = (int)m; K = (int)k; N = (int)n;
        shape.assign(x->sizes().begin(), x->sizes().end());
        shape.back() = n;
        return row_stride(x, x->sizes(), type, dev, 1, sx) && row_stride(weight, {n, k}, type, dev, 1, sw) &&
               c10::cuda::current_device() == dev;
    }
};

// (kda_linear_fwd, kda_linear_copies, kda_linear_fwd_workspace_bytes, x, weight, bias, residual,
//  activation, save)
PyObject *linear_fwd(PyObject *const *a) {
    Linear l;
    const Tensor *bias, *residual;
    kda_linear_fwd_opts_t op = {};
    if (!l.read(a[3], a[4], a[7]) || !optional(a[5], bias) || !optional(a[6], residual) ||
        (bias && !fits(bias, {l.N}, l.type, l.dev)) ||
        (residual && !row_stride(residual, l.shape, l.type, l.dev, 1, op.residual_stride)))
        Py_RETURN_NONE;
    const int save = PyObject_IsTrue(a[8]);
    if (save < 0) return nullptr;
    Tensor out[2] = {empty(l.shape, l.type, *l.x)};
    if (save && l.act != KDA_ACT_NONE) {
        out[1] = empty(l.shape, l.type, *l.x);
        op.saved = out[1].data_ptr();
    }
    op.bias = address(bias);
    op.residual = address(residual);
    op.activation = l.act;
    op.x_stride = l.sx;
    op.weight_stride = l.sw;
    const int copies = function<decltype(&kda_linear_copies)>(a[1])(l.x->data_ptr(), l.sx, l.weight->data_ptr(),
                                                                    l.sw, nullptr, 0);
    op.workspace_bytes = function<decltype(&kda_linear_fwd_workspace_bytes)>(a[2])(l.M, l.K, l.N, copies);
    Tensor work;
    if (op.workspace_bytes) {
        work = bytes(op.workspace_bytes, *l.x);
        op.workspace = work.data_ptr();
    }
    const kda_stream_t stream = stream_of(l.dev);
    if (!call([&] {
            return function<decltype(&kda_linear_fwd)>(a[0])(l.x->data_ptr(), l.weight->data_ptr(),
                                                             out[0].data_ptr(), l.M, l.K, l.N, l.dtype, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// (kda_linear_bwd, kda_linear_copies, kda_linear_bwd_workspace_bytes, dy, x, weight, saved, activation,
//  input_grad, weight_grad, bias_grad)
PyObject *linear_bwd(PyObject *const *a) {
    Linear l;
    const Tensor *dy = tensor(a[3]), *saved;
    kda_linear_bwd_opts_t op = {};
    if (!l.read(a[4], a[5], a[7]) || !optional(a[6], saved) ||
        !row_stride(dy, l.shape, l.type, l.dev, 1, op.dy_stride) ||
        (l.act != KDA_ACT_NONE && (!saved || !fits(saved, l.shape, l.type, l.dev))))
        Py_RETURN_NONE;
    int wanted = 0;
    for (int i = 0; i < 3; ++i) {
        const int on = PyObject_IsTrue(a[8 + i]);
        if (on < 0) return nullptr;
        wanted |= on << i;
    }
    Tensor out[3];
    if (wanted & KDA_GRAD_X) out[0] = empty(l.x->sizes(), l.type, *l.x);
    if (wanted & KDA_GRAD_WEIGHT) out[1] = empty({l.N, l.K}, l.type, *l.x);
    if (wanted & KDA_GRAD_BIAS) out[2] = empty({l.N}, l.type, *l.x);
    auto to = [](const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
    op.saved = l.act != KDA_ACT_NONE ? address(saved) : nullptr;
    op.activation = l.act;
    op.x_stride = l.sx;
    op.weight_stride = l.sw;
    const int copies = function<decltype(&kda_linear_copies)>(a[1])(
        l.x->data_ptr(), l.sx, l.weight->data_ptr(), l.sw, dy->data_ptr(), op.dy_stride);
    op.workspace_bytes =
        function<decltype(&kda_linear_bwd_workspace_bytes)>(a[2])(l.M, l.K, l.N, l.act, copies, wanted);
    Tensor work;
    if (op.workspace_bytes) {
        work = bytes(op.workspace_bytes, *l.x);
        op.workspace = work.data_ptr();
    }
    const kda_stream_t stream = stream_of(l.dev);
    if (!call([&] {
            return function<decltype(&kda_linear_bwd)>(a[0])(dy->data_ptr(), l.x->data_ptr(), l.weight->data_ptr(),
                                                             to(out[0]), to(out[1]), to(out[2]), l.M, l.K, l.N,
                                                             l.dtype, &op, stream);
        }))
        Py_RETURN_NONE;
    return wrap_all(out);
}

// The function with its number of arguments checked; a C++ exception (out of memory, ...) leaves
// the call to the Python side, which meets and reports it itself.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *method(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const std::exception &) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

#define METHOD(name, n) {#name, (PyCFunction)(void *)method<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(step, 10),          METHOD(chunk_fwd, 11),
                         METHOD(chunk_bwd, 11),     METHOD(layer_norm_fwd, 5),
                         METHOD(layer_norm_bwd, 7), METHOD(conv_fwd, 8),
                         METHOD(conv_bwd, 8),       METHOD(conv_step, 7),
                         METHOD(scan_fwd, 15),      METHOD(scan_bwd, 14),
                         METHOD(scan_step, 11),     METHOD(linear_fwd, 9),
                         METHOD(linear_bwd, 11),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                      nullptr,               nullptr,   nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
