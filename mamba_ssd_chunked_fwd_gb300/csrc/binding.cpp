// binding.cpp -- the Python side of the selective scan, its convolution and the
// block norm, in C++: checks torch tensors, fills the C structures of
// include/ssd.h, allocates outputs and workspaces with torch, and calls the
// library on the stream it is given.  A single-token call takes a few
// microseconds on the GPU; the same checks in Python take ten.
//
// Each function takes its arguments by position (selective.py has the
// signatures), raises ValueError for what the binding cannot express, and
// returns the result, or the library's status as an int when that is not 0.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <dlfcn.h>

#include <sstream>
#include <stdexcept>

#include "ssd.h"

namespace {

#define SSD_ENTRIES(X)                       \
    X(ssd_selective_scan_workspace_size)     \
    X(ssd_selective_scan)                    \
    X(ssd_selective_scan_bwd_workspace_size) \
    X(ssd_selective_scan_bwd)                \
    X(ssd_selective_scan_step)               \
    X(ssd_causal_conv_carry)                 \
    X(ssd_causal_conv_bwd_workspace_size)    \
    X(ssd_causal_conv_bwd)                   \
    X(ssd_causal_conv_step)                  \
    X(ssd_block_norm)                        \
    X(ssd_block_norm_bwd_workspace_size)     \
    X(ssd_block_norm_bwd)

#define X(name) decltype(&::name) p_##name = nullptr;
SSD_ENTRIES(X)
#undef X

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

template <class... T>
[[noreturn]] void refuse(const T &...parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw Refused(s.str());
}

// A tensor argument; None gives nullptr.
const Tensor *tensor(PyObject *o, const char *what) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(what, ": not a tensor");
    return &THPVariable_Unpack(o);
}
const Tensor &needed(PyObject *o, const char *what) {
    const Tensor *t = tensor(o, what);
    if (!t) refuse(what, " is required");
    return *t;
}

int32_t code_of(ScalarType t, const char *what) {
    if (t == at::kFloat) return SSD_F32;
    if (t == at::kHalf) return SSD_F16;
    if (t == at::kBFloat16) return SSD_BF16;
    refuse(what, ": unsupported dtype ", t);
}

void fits(const Tensor &t, IntArrayRef shape, ScalarType type, int64_t dev, const char *what) {
    if (t.sizes() != shape) refuse(what, ": shape ", t.sizes(), ", expected ", shape);
    if (t.scalar_type() != type) refuse(what, ": dtype ", t.scalar_type(), ", expected ", type);
    if (!t.is_cuda() || t.get_device() != dev) refuse(what, ": on ", t.device(), ", expected CUDA device ", dev);
}

// The address of a dense tensor of this shape and type.
template <class P = void>
P *dense(const Tensor *t, IntArrayRef shape, ScalarType type, int64_t dev, const char *what) {
    if (!t) return nullptr;
    fits(*t, shape, type, dev, what);
    if (!t->is_contiguous()) refuse(what, ": must be contiguous");
    return static_cast<P *>(t->data_ptr());
}

bool inner_dense(const Tensor &t, int64_t lead) {
    int64_t want = 1;
    for (int64_t i = t.dim() - 1; i >= lead; --i) {
        if (t.size(i) != 1 && t.stride(i) != want) return false;
        want *= t.size(i);
    }
    return true;
}

// A [B,L,...] tensor whose tokens are dense.
const void *tokens(const Tensor *t, IntArrayRef shape, ScalarType type, int64_t dev, const char *what, int64_t (&st)[2]) {
    st[0] = st[1] = 0;
    if (!t) return nullptr;
    fits(*t, shape, type, dev, what);
    if (t->is_contiguous()) return t->data_ptr();
    if (!inner_dense(*t, 2)) refuse(what, ": the values of a token must be contiguous");
    st[0] = t->size(0) == 1 ? 0 : t->stride(0);
    st[1] = t->size(1) == 1 ? 0 : t->stride(1);
    if (st[0] == 0 && st[1] == 0 && t->numel()) {
        if (t->size(1) != 1) refuse(what, ": broadcast over every token");
        // one token for every sequence; its stride leads nowhere, and two zeros would mean dense
        st[1] = t->numel() / t->size(0);
    }
    return t->data_ptr();
}

// A [B,...] tensor whose rows are dense.
const void *rows(const Tensor *t, IntArrayRef shape, ScalarType type, int64_t dev, const char *what, int64_t &row) {
    row = 0;
    if (!t) return nullptr;
    fits(*t, shape, type, dev, what);
    if (t->is_contiguous()) return t->data_ptr();
    if (!inner_dense(*t, 1)) refuse(what, ": the values of a row must be contiguous");
    if (t->size(0) == 1) return t->data_ptr();
    if (t->stride(0) <= 0) refuse(what, ": rows must be apart");
    row = t->stride(0);
    return t->data_ptr();
}

void ndim(const Tensor &t, int64_t n, const char *what) {
    if (t.dim() != n) refuse(what, ": ", t.dim(), " dimensions, expected ", n);
}

int64_t cuda_device(const Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(name, " takes CUDA tensors");
    return t.get_device();
}

Tensor fresh(IntArrayRef shape, const Tensor &like, ScalarType type) { return at::empty(shape, like.options().dtype(type)); }
Tensor fresh(IntArrayRef shape, const Tensor &like) { return fresh(shape, like, like.scalar_type()); }
Tensor like(const Tensor &t) { return fresh(t.sizes(), t); }

// An output: the caller's tensor, or a new one.
Tensor output(PyObject *o, IntArrayRef shape, const Tensor &x, ScalarType type, int64_t dev, const char *what) {
    const Tensor *t = tensor(o, what);
    if (!t) return fresh(shape, x, type);
    dense(t, shape, type, dev, what);
    return *t;
}

Tensor workspace(size_t bytes, const Tensor &x) {
    return bytes ? at::empty({(int64_t)bytes}, x.options().dtype(at::kByte)) : Tensor();
}

ScalarType step_type(const Tensor &x, const Tensor &dt) {
    if (dt.scalar_type() != x.scalar_type() && dt.scalar_type() != at::kFloat)
        refuse("dt: dtype ", dt.scalar_type(), ", expected ", x.scalar_type(), " or Float");
    return dt.scalar_type();
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused("");
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused("");
    return v != 0;
}
void *stream_of(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused("");
    return p;
}

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *status(ssd_status st) { return PyLong_FromLong((long)st); }
PyObject *pair(PyObject *a, PyObject *b) {
    PyObject *r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}
// Takes the tensor into the dict.
void put(PyObject *d, const char *k, const Tensor &t) {
    PyObject *o = wrap(t);
    if (!o || PyDict_SetItemString(d, k, o) < 0) {
        Py_XDECREF(o);
        throw Refused("");
    }
    Py_DECREF(o);
}
struct Dict {
    PyObject *d = PyDict_New();
    ~Dict() { Py_XDECREF(d); }
    PyObject *release() {
        PyObject *r = d;
        d = nullptr;
        return r;
    }
};

// ---- selective scan

// x, dt, A, B, C, dt_softplus, dt_min, dt_max, D, z, dt_bias, initial_states, lengths
void scan_args(PyObject *const *a, const char *name, ssd_scan_args &p) {
    const Tensor &x = needed(a[0], "x"), &dt = needed(a[1], "dt"), &A = needed(a[2], "A"), &B = needed(a[3], "B"),
                 &C = needed(a[4], "C");
    const int64_t dev = cuda_device(x, name);
    ndim(x, 3, "x"), ndim(B, 4, "B"), ndim(A, 2, "A");
    p = ssd_scan_args{};
    p.B = x.size(0), p.L = x.size(1), p.D = x.size(2), p.G = B.size(2), p.N = B.size(3);
    const ScalarType io = x.scalar_type(), f32 = at::kFloat, td = step_type(x, dt);
    p.x_dtype = code_of(io, "x"), p.dt_dtype = code_of(td, "dt");
    const int64_t bc[4] = {p.B, p.L, p.G, p.N}, state[3] = {p.B, p.D, p.N}, an[2] = {p.D, p.N};
    p.x = tokens(&x, x.sizes(), io, dev, "x", p.x_stride);
    p.dt = tokens(&dt, x.sizes(), td, dev, "dt", p.dt_stride);
    p.Bm = tokens(&B, bc, io, dev, "B", p.b_stride);
    p.Cm = tokens(&C, bc, io, dev, "C", p.c_stride);
    p.z = tokens(tensor(a[9], "z"), x.sizes(), io, dev, "z", p.z_stride);
    p.A = dense<float>(&A, an, f32, dev, "A");
    p.Dskip = dense<float>(tensor(a[8], "D"), {p.D}, f32, dev, "D");
    p.dt_bias = dense<float>(tensor(a[10], "dt_bias"), {p.D}, f32, dev, "dt_bias");
    p.initial_state = dense<float>(tensor(a[11], "initial_states"), state, f32, dev, "initial_states");
    p.lengths = dense<int32_t>(tensor(a[12], "lengths"), {p.B}, at::kInt, dev, "lengths");
    p.dt_softplus = truth(a[5]);
    p.dt_min = (float)number(a[6]), p.dt_max = (float)number(a[7]);
}

// stream, the scan's 13, return_final_state, out
PyObject *selective_scan(PyObject *const *a) {
    ssd_scan_args p;
    scan_args(a + 1, "selective_scan", p);
    const Tensor &x = needed(a[1], "x");
    const bool want = truth(a[14]);
    Tensor y = output(a[15], x.sizes(), x, x.scalar_type(), x.get_device(), "out"), fin;
    p.y = y.data_ptr();
    if (want) {
        fin = fresh({p.B, p.D, p.N}, x, at::kFloat);
        p.final_state = fin.data_ptr<float>();
    }
    size_t bytes = 0;
    ssd_status st = p_ssd_selective_scan_workspace_size(&p, &bytes);
    if (st != SSD_OK) return status(st);
    const Tensor ws = workspace(bytes, x);
    if (bytes) p.workspace = ws.data_ptr(), p.workspace_bytes = bytes;
    if ((st = p_ssd_selective_scan(&p, stream_of(a[0]))) != SSD_OK) return status(st);
    return want ? pair(wrap(y), wrap(fin)) : wrap(y);
}

// stream, the scan's 13, dy, dfinal, want_dh0 (None: with initial_states)
PyObject *selective_scan_bwd(PyObject *const *a) {
    ssd_scan_bwd_args b = {};
    scan_args(a + 1, "selective_scan_bwd", b.fwd);
    const ssd_scan_args &p = b.fwd;
    const Tensor &x = needed(a[1], "x"), &dt = needed(a[2], "dt"), &dy = needed(a[14], "dy");
    const int64_t dev = x.get_device(), state[3] = {p.B, p.D, p.N};
    b.dy = dense(&dy, x.sizes(), x.scalar_type(), dev, "dy");
    b.dfinal = dense<float>(tensor(a[15], "dfinal"), state, at::kFloat, dev, "dfinal");
    Dict d;
    auto out = [&](const char *k, IntArrayRef shape, ScalarType type) {
        Tensor t = fresh(shape, x, type);
        put(d.d, k, t);
        return t.data_ptr();
    };
    const int64_t bc[4] = {p.B, p.L, p.G, p.N}, an[2] = {p.D, p.N};
    const ScalarType io = x.scalar_type(), f32 = at::kFloat;
    b.dx = out("dx", x.sizes(), io);
    b.ddt = out("ddt", x.sizes(), dt.scalar_type());
    b.dA = static_cast<float *>(out("dA", an, f32));
    b.dB = out("dB", bc, io);
    b.dC = out("dC", bc, io);
    if (p.Dskip) b.dD = static_cast<float *>(out("dD", {p.D}, f32));
    if (p.z) b.dz = out("dz", x.sizes(), io);
    if (p.dt_bias) b.ddt_bias = static_cast<float *>(out("ddt_bias", {p.D}, f32));
    if (a[16] == Py_None ? p.initial_state != nullptr : truth(a[16])) b.dh0 = static_cast<float *>(out("dh0", state, f32));
    size_t bytes = 0;
    ssd_status st = p_ssd_selective_scan_bwd_workspace_size(&b, &bytes);
    if (st != SSD_OK) return status(st);
    const Tensor ws = workspace(bytes, x);
    b.workspace = ws.data_ptr(), b.workspace_bytes = bytes;
    if ((st = p_ssd_selective_scan_bwd(&b, stream_of(a[0]))) != SSD_OK) return status(st);
    return d.release();
}

// stream, x, dt, A, B, C, state, dt_softplus, dt_min, dt_max, state_out, slots, D, z, dt_bias, out
PyObject *selective_scan_step(PyObject *const *a) {
    const Tensor &x = needed(a[1], "x"), &dt = needed(a[2], "dt"), &A = needed(a[3], "A"), &B = needed(a[4], "B"),
                 &C = needed(a[5], "C"), &state = needed(a[6], "state");
    const int64_t dev = cuda_device(x, "selective_scan_step");
    ndim(x, 2, "x"), ndim(B, 3, "B"), ndim(state, 3, "state"), ndim(A, 2, "A");
    ssd_scan_step_args p = {};
    p.B = x.size(0), p.D = x.size(1), p.G = B.size(1), p.N = B.size(2), p.nslots = state.size(0);
    const ScalarType io = x.scalar_type(), f32 = at::kFloat, td = step_type(x, dt);
    p.x_dtype = code_of(io, "x"), p.dt_dtype = code_of(td, "dt");
    const int64_t bc[3] = {p.B, p.G, p.N}, pool[3] = {p.nslots, p.D, p.N}, an[2] = {p.D, p.N};
    p.x = rows(&x, x.sizes(), io, dev, "x", p.x_row);
    p.dt = rows(&dt, x.sizes(), td, dev, "dt", p.dt_row);
    p.Bm = rows(&B, bc, io, dev, "B", p.b_row);
    p.Cm = rows(&C, bc, io, dev, "C", p.c_row);
    p.z = rows(tensor(a[13], "z"), x.sizes(), io, dev, "z", p.z_row);
    p.A = dense<float>(&A, an, f32, dev, "A");
    p.Dskip = dense<float>(tensor(a[12], "D"), {p.D}, f32, dev, "D");
    p.dt_bias = dense<float>(tensor(a[14], "dt_bias"), {p.D}, f32, dev, "dt_bias");
    float *s = dense<float>(&state, pool, f32, dev, "state"), *so = dense<float>(tensor(a[10], "state_out"), pool, f32, dev, "state_out");
    p.state = s, p.state_out = so ? so : s;
    p.slots = dense<int32_t>(tensor(a[11], "slots"), {p.B}, at::kInt, dev, "slots");
    p.dt_softplus = truth(a[7]);
    p.dt_min = (float)number(a[8]), p.dt_max = (float)number(a[9]);
    Tensor y = output(a[15], x.sizes(), x, io, dev, "out");
    p.y = y.data_ptr();
    const ssd_status st = p_ssd_selective_scan_step(&p, stream_of(a[0]));
    return st != SSD_OK ? status(st) : wrap(y);
}

// ---- convolution

// x, w, bias, silu, initial_state, lengths
void conv_args(PyObject *const *a, const char *name, ssd_conv_args &p) {
    const Tensor &x = needed(a[0], "x"), &w = needed(a[1], "w");
    const int64_t dev = cuda_device(x, name);
    ndim(x, 3, "x"), ndim(w, 2, "w");
    p = ssd_conv_args{};
    p.B = x.size(0), p.L = x.size(1), p.C = x.size(2), p.W = w.size(1);
    const ScalarType io = x.scalar_type(), f32 = at::kFloat;
    p.dtype = code_of(io, "x");
    const int64_t cw[2] = {p.C, p.W}, state[3] = {p.B, p.W - 1, p.C};
    p.x = tokens(&x, x.sizes(), io, dev, "x", p.x_stride);
    p.w = dense<float>(&w, cw, f32, dev, "w");
    p.bias = dense<float>(tensor(a[2], "bias"), {p.C}, f32, dev, "bias");
    p.silu = truth(a[3]);
    p.initial_state = dense(tensor(a[4], "initial_state"), state, io, dev, "initial_state");
    p.lengths = dense<int32_t>(tensor(a[5], "lengths"), {p.B}, at::kInt, dev, "lengths");
}

// stream, the convolution's 6, return_final_state, out
PyObject *causal_conv1d_carry(PyObject *const *a) {
    ssd_conv_args p;
    conv_args(a + 1, "causal_conv1d_carry", p);
    const Tensor &x = needed(a[1], "x");
    const bool want = truth(a[7]);
    Tensor y = output(a[8], x.sizes(), x, x.scalar_type(), x.get_device(), "out"), fin;
    p.y = y.data_ptr();
    if (want) {
        fin = fresh({p.B, p.W - 1, p.C}, x);
        p.final_state = fin.data_ptr();
    }
    const ssd_status st = p_ssd_causal_conv_carry(&p, stream_of(a[0]));
    if (st != SSD_OK) return status(st);
    return want ? pair(wrap(y), wrap(fin)) : wrap(y);
}

// stream, the convolution's 6, dy, dfinal, want_dh0 (None: with initial_state)
PyObject *causal_conv1d_bwd(PyObject *const *a) {
    ssd_conv_bwd_args b = {};
    conv_args(a + 1, "causal_conv1d_bwd", b.fwd);
    const ssd_conv_args &p = b.fwd;
    const Tensor &x = needed(a[1], "x"), &w = needed(a[2], "w"), &dy = needed(a[7], "dy");
    const int64_t dev = x.get_device(), state[3] = {p.B, p.W - 1, p.C};
    b.dy = dense(&dy, x.sizes(), x.scalar_type(), dev, "dy");
    b.dfinal = dense(tensor(a[8], "dfinal"), state, x.scalar_type(), dev, "dfinal");
    Dict d;
    auto out = [&](const char *k, Tensor t) {
        put(d.d, k, t);
        return t.data_ptr();
    };
    b.dx = out("dx", fresh(x.sizes(), x));
    b.dw = static_cast<float *>(out("dw", like(w)));
    if (p.bias) b.dbias = static_cast<float *>(out("dbias", fresh({p.C}, x, at::kFloat)));
    if (a[9] == Py_None ? p.initial_state != nullptr || tensor(a[5], "initial_state") != nullptr : truth(a[9]))
        b.dh0 = out("dh0", fresh(state, x));
    size_t bytes = 0;
    ssd_status st = p_ssd_causal_conv_bwd_workspace_size(&b, &bytes);
    if (st != SSD_OK) return status(st);
    const Tensor ws = workspace(bytes, x);
    b.workspace = ws.data_ptr(), b.workspace_bytes = bytes;
    if ((st = p_ssd_causal_conv_bwd(&b, stream_of(a[0]))) != SSD_OK) return status(st);
    return d.release();
}

// stream, x, state, w, bias, silu, state_out, slots, out
PyObject *causal_conv1d_step(PyObject *const *a) {
    const Tensor &x = needed(a[1], "x"), &state = needed(a[2], "state"), &w = needed(a[3], "w");
    const int64_t dev = cuda_device(x, "causal_conv1d_step");
    ndim(x, 2, "x"), ndim(w, 2, "w"), ndim(state, 3, "state");
    ssd_conv_step_args p = {};
    p.B = x.size(0), p.C = x.size(1), p.W = w.size(1), p.nslots = state.size(0);
    const ScalarType io = x.scalar_type(), f32 = at::kFloat;
    p.dtype = code_of(io, "x");
    const int64_t cw[2] = {p.C, p.W}, pool[3] = {p.nslots, p.W - 1, p.C};
    p.x = rows(&x, x.sizes(), io, dev, "x", p.x_row);
    p.w = dense<float>(&w, cw, f32, dev, "w");
    p.bias = dense<float>(tensor(a[4], "bias"), {p.C}, f32, dev, "bias");
    void *s = dense(&state, pool, io, dev, "state");
    const Tensor *to = tensor(a[6], "state_out");
    p.state = s, p.state_out = to ? dense(to, pool, io, dev, "state_out") : s;
    p.slots = dense<int32_t>(tensor(a[7], "slots"), {p.B}, at::kInt, dev, "slots");
    p.silu = truth(a[5]);
    Tensor y = output(a[8], x.sizes(), x, io, dev, "out");
    p.y = y.data_ptr();
    const ssd_status st = p_ssd_causal_conv_step(&p, stream_of(a[0]));
    return st != SSD_OK ? status(st) : wrap(y);
}

// ---- block norm

// o, r, w_pre, w_post, gate, scale, eps; io: the block's type
void norm_args(PyObject *const *a, const Tensor &r, ScalarType io, ssd_block_norm_args &p) {
    const int64_t dev = r.get_device();
    if (r.dim() < 1) refuse("r: at least one dimension");
    const ScalarType f32 = at::kFloat;
    p = ssd_block_norm_args{};
    p.D = r.size(-1);
    p.rows = p.D ? r.numel() / p.D : 0;
    p.rows_per_gate = 1;
    p.dtype = code_of(io, "o"), p.stream_dtype = code_of(r.scalar_type(), "r");
    p.o = dense(tensor(a[0], "o"), r.sizes(), io, dev, "o");
    if (const Tensor *g = tensor(a[4], "gate")) {
        if (g->sizes() != r.sizes()) {  // [B, D] for [B, ..., D]
            if (r.dim() < 2 || g->dim() != 2 || g->size(0) != r.size(0) || g->size(1) != p.D)
                refuse("gate: shape ", g->sizes(), ", expected ", r.sizes(), " or [", r.dim() < 2 ? 0 : r.size(0), ", ", p.D, "]");
            p.rows_per_gate = r.size(0) ? p.rows / r.size(0) : 0;
        }
        p.gate = dense(g, g->sizes(), io, dev, "gate");
    }
    p.w_pre = dense<float>(&needed(a[2], "w_pre"), {p.D}, f32, dev, "w_pre");
    p.w_post = dense<float>(tensor(a[3], "w_post"), {p.D}, f32, dev, "w_post");
    p.scale = dense<float>(tensor(a[5], "scale"), {p.D}, f32, dev, "scale");
    p.eps = (float)number(a[6]);
}

// stream, the norm's 7, like (a tensor of n's type, used without o), out, r_out
PyObject *block_norm(PyObject *const *a) {
    const Tensor &r = needed(a[2], "r");
    const int64_t dev = cuda_device(r, "block_norm");
    const Tensor *o = tensor(a[1], "o"), *n_like = tensor(a[8], "like");
    const ScalarType io = o ? o->scalar_type() : n_like ? n_like->scalar_type() : r.scalar_type();
    ssd_block_norm_args p;
    norm_args(a + 1, r, io, p);
    p.r = dense(&r, r.sizes(), r.scalar_type(), dev, "r");
    Tensor n = output(a[9], r.sizes(), r, io, dev, "out"), r_out = r;
    p.n = n.data_ptr();
    if (o) {
        r_out = output(a[10], r.sizes(), r, r.scalar_type(), dev, "r_out");
        p.r_out = r_out.data_ptr();
    }
    const ssd_status st = p_ssd_block_norm(&p, stream_of(a[0]));
    if (st != SSD_OK) return status(st);
    PyObject *second = o ? wrap(r_out) : a[2];
    if (!o) Py_INCREF(second);
    return pair(wrap(n), second);
}

// stream, the norm's 7 (r: the stored r'), dn, dr_out
PyObject *block_norm_bwd(PyObject *const *a) {
    const Tensor &r = needed(a[2], "r_out"), &dn = needed(a[8], "dn");
    const int64_t dev = cuda_device(dn, "block_norm_bwd");
    if (!r.is_cuda()) refuse("block_norm_bwd takes CUDA tensors");
    ssd_block_norm_bwd_args b = {};
    norm_args(a + 1, r, dn.scalar_type(), b.fwd);
    ssd_block_norm_args &p = b.fwd;
    p.r_out = dense(&r, r.sizes(), r.scalar_type(), dev, "r_out");
    b.dn = dense(&dn, r.sizes(), dn.scalar_type(), dev, "dn");
    b.dr_out = dense(tensor(a[9], "dr_out"), r.sizes(), r.scalar_type(), dev, "dr_out");
    Dict d;
    auto out = [&](const char *k, const Tensor &t) {
        Tensor n = like(t);
        put(d.d, k, n);
        return n.data_ptr();
    };
    b.dr = out("dr", r);
    b.dw_pre = static_cast<float *>(out("dw_pre", needed(a[3], "w_pre")));
    if (const Tensor *o = tensor(a[1], "o")) b.d_o = out("do", *o);
    if (const Tensor *t = tensor(a[4], "w_post")) b.dw_post = static_cast<float *>(out("dw_post", *t));
    if (const Tensor *t = tensor(a[5], "gate")) b.dgate = out("dgate", *t);
    if (const Tensor *t = tensor(a[6], "scale")) b.dscale = static_cast<float *>(out("dscale", *t));
    size_t bytes = 0;
    ssd_status st = p_ssd_block_norm_bwd_workspace_size(&b, &bytes);
    if (st != SSD_OK) return status(st);
    const Tensor ws = workspace(bytes, r);
    b.workspace = ws.data_ptr(), b.workspace_bytes = bytes;
    if ((st = p_ssd_block_norm_bwd(&b, stream_of(a[0]))) != SSD_OK) return status(st);
    return d.release();
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, N);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// Resolves the library's entries.
PyObject *load(PyObject *, PyObject *path) {
    const char *s = PyUnicode_AsUTF8(path);
    if (!s) return nullptr;
    void *h = dlopen(s, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
        PyErr_SetString(PyExc_OSError, dlerror());
        return nullptr;
    }
#define X(name)                                                         \
    p_##name = reinterpret_cast<decltype(&::name)>(dlsym(h, #name));    \
    if (!p_##name) {                                                    \
        PyErr_SetString(PyExc_OSError, "missing entry " #name);         \
        return nullptr;                                                 \
    }
    SSD_ENTRIES(X)
#undef X
    Py_RETURN_NONE;
}

#define M(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"load", load, METH_O, nullptr},
                         M(selective_scan, 16),
                         M(selective_scan_bwd, 17),
                         M(selective_scan_step, 16),
                         M(causal_conv1d_carry, 9),
                         M(causal_conv1d_bwd, 10),
                         M(causal_conv1d_step, 9),
                         M(block_norm, 11),
                         M(block_norm_bwd, 10),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ssd_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ssd_binding(void) { return PyModule_Create(&module); }
