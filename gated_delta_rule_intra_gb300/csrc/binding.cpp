// The short way from Python to the recurrence, single-token and layer-norm entry points: checks
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
                         METHOD(layer_norm_bwd, 7), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                      nullptr,               nullptr,   nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
