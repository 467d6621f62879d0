// The operators around the scan, linear attention and beam search as functions on torch tensors: checks of the arguments,
// allocation of what the caller did not bring, and the call into libssd.so on the current
// stream.  A CPython module rather than a ctypes binding because the smallest calls (a
// handful of rows, one token) spend longer in the host code than on the GPU: a call costs
// about a third of what the same steps take in Python.
//
// Positional arguments only; the Python modules `layer`, `attention` and `beam` have the signatures
// and document them.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "ssd.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // SSDError

struct Err {
    PyObject* type;
    std::string text;
};
struct Status {
    int code;
    const char* where;
};
struct Raised {};  // a Python error is already set

[[noreturn]] void value_error(const std::string& s) { throw Err{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw Err{PyExc_TypeError, s}; }

void ok(ssd_status_t s, const char* where) {
    if (s != SSD_OK) throw Status{s, where};
}

std::string text(at::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}
std::string text(at::ScalarType t) {
    return t == at::kFloat      ? "torch.float32"
           : t == at::kBFloat16 ? "torch.bfloat16"
           : t == at::kInt      ? "torch.int32"
                                : std::string(c10::toString(t));
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
// None or a tensor.
const Tensor* maybe(PyObject* o, const char* name) {
    return o == Py_None ? nullptr : &tensor(o, name);
}
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

void on_device(const Tensor& t, const char* name, at::Device dev) {
    if (t.device() != dev)
        value_error(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
}
void of_type(const Tensor& t, const char* name, at::ScalarType type) {
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + text(type) + ", got " + text(t.scalar_type()));
}
void of_shape(const Tensor& t, const char* name, at::IntArrayRef shape) {
    if (t.sizes() != shape)
        value_error(std::string(name) + " must be " + text(shape) + ", got " + text(t.sizes()));
}
void contiguous(const Tensor& t, const char* name) {
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}
void check(const Tensor& t, const char* name, at::Device dev, at::ScalarType type,
           at::IntArrayRef shape) {
    on_device(t, name, dev);
    of_type(t, name, type);
    of_shape(t, name, shape);
    contiguous(t, name);
}
int code(const Tensor& t, const char* name) {
    if (t.scalar_type() == at::kFloat) return SSD_DTYPE_F32;
    if (t.scalar_type() == at::kBFloat16) return SSD_DTYPE_BF16;
    type_error(std::string(name) + " must be float32 or bfloat16, got " + text(t.scalar_type()));
}
void on_gpu(const Tensor& t, const char* name) {
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
}

// The stride between the rows of t (its last dimension's vectors), which must be evenly
// spaced and must not overlap; the last dimension itself must be contiguous.
int64_t rows(const Tensor& t, const char* name) {
    const int64_t d = t.dim();
    if (d < 1) value_error(std::string(name) + " must have a last dimension");
    const auto size = t.sizes(), stride = t.strides();
    const int64_t last = size[d - 1];
    if (t.is_contiguous()) return last;
    if (last > 1 && stride[d - 1] != 1)
        value_error(std::string(name) + ": neighbouring channels must be adjacent");
    int64_t step = -1, span = 1;
    for (int64_t i = d - 2; i >= 0; --i) {
        if (size[i] == 1) continue;
        if (step < 0)
            step = stride[i];
        else if (stride[i] != span * step)
            value_error(std::string(name) + ": rows must be evenly spaced");
        span *= size[i];
    }
    if (step < 0) return last;
    if (step < last) value_error(std::string(name) + ": rows overlap");
    return step;
}
int64_t rows(const Tensor& t, const char* name, at::Device dev, at::ScalarType type,
             at::IntArrayRef shape) {
    on_device(t, name, dev);
    of_type(t, name, type);
    of_shape(t, name, shape);
    return rows(t, name);
}

Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    return Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}

// The given output, checked by the caller, or a new one.
Tensor brought(PyObject* dict, const char* key) {
    if (dict == Py_None) return Tensor();
    PyObject* o = PyDict_GetItemString(dict, key);
    return o && o != Py_None ? tensor(o, key) : Tensor();
}

// Workspace: the given tensor, or a new one of n bytes.
struct Scratch {
    Tensor t;
    void* p;
    size_t n;
    Scratch(PyObject* o, size_t need, at::Device dev) {
        if (o == Py_None) {
            t = empty({(int64_t)need}, at::kByte, dev);
        } else {
            t = tensor(o, "workspace");
            on_device(t, "workspace", dev);
            contiguous(t, "workspace");
            if (t.nbytes() < need)
                value_error("workspace too small: need " + std::to_string(need) + " bytes");
        }
        p = t.data_ptr();
        n = t.nbytes();
    }
};

void* stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

struct Dict {
    PyObject* d;
    explicit Dict(PyObject* given) {
        if (given == Py_None) {
            d = PyDict_New();
        } else {
            if (!PyDict_Check(given)) type_error("out must be a dict");
            d = given;
            Py_INCREF(d);
        }
        if (!d) throw Raised();
    }
    ~Dict() { Py_XDECREF(d); }
    void set(const char* key, const Tensor& t) {
        PyObject* o = THPVariable_Wrap(t);
        if (!o || PyDict_SetItemString(d, key, o) < 0) {
            Py_XDECREF(o);
            throw Raised();
        }
        Py_DECREF(o);
    }
    PyObject* release() {
        PyObject* r = d;
        d = nullptr;
        return r;
    }
};
PyObject* wrap(const Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    PyObject* o = THPVariable_Wrap(t);
    if (!o) throw Raised();
    return o;
}
// Steals the references; none may be null.
PyObject* tuple(std::initializer_list<PyObject*> items) {
    PyObject* r = PyTuple_New((Py_ssize_t)items.size());
    if (!r) throw Raised();
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
    return r;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}
long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
int32_t int32(PyObject* o, const char* name) {
    const long long v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
    return (int32_t)v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v != 0;
}

// ------------------------------------------------------------------ convolution
// Up to three pieces of the channels, each with a shape of its own.
struct Pieces {
    int n = 0;
    c10::SmallVector<int64_t, 6> shape[3];  // [batch, L, ...]
    int64_t channels[3] = {0, 0, 0};
    void add(int64_t batch, int64_t L) {
        if (n == 3) value_error("split must name one to three pieces");
        shape[n] = {batch, L};
        channels[n++] = 1;
    }
    void dim(int64_t d) {
        if (d < 1) value_error("split sizes must be positive");
        shape[n - 1].push_back(d);
        channels[n - 1] *= d;
    }
    void total(int64_t C) const {
        const int64_t s = channels[0] + channels[1] + channels[2];
        if (s != C)
            value_error("split adds up to " + std::to_string(s) + " channels, u has " +
                        std::to_string(C));
    }
};

struct ConvCall {
    ssd_conv_t p;
    int64_t n, width, C;
};
void conv_problem(ConvCall* c, const Tensor& u, const Tensor& w, const Tensor* b, const Pieces& s,
                  bool silu, const Tensor* cu, const Tensor* pos, const Tensor* init) {
    const auto dev = u.device();
    const int64_t stride = rows(u, "u");
    c->C = u.size(2);
    if (w.dim() != 2 || w.size(0) != c->C) value_error("weight must be [channels, width]");
    c->width = w.size(1);
    const int wcode = code(w, "weight");
    on_device(w, "weight", dev);
    contiguous(w, "weight");
    if (b) check(*b, "bias", dev, w.scalar_type(), {c->C});
    int64_t nseq = 0;
    if (cu) {
        on_device(*cu, "cu_seqlens", dev);
        of_type(*cu, "cu_seqlens", at::kInt);
        contiguous(*cu, "cu_seqlens");
        if (u.size(0) != 1) value_error("packed sequences need batch == 1");
        nseq = cu->numel() - 1;
        if (cu->dim() != 1 || nseq < 1) value_error("cu_seqlens must be [nseq + 1]");
    }
    c->n = nseq ? nseq : u.size(0);
    if (pos) check(*pos, "positions", dev, at::kInt, {c->n});
    if (init) check(*init, "initial_state", dev, u.scalar_type(), {c->n, c->width, c->C});
    c->p = {};
    c->p.batch = u.size(0);
    c->p.seqlen = u.size(1);
    c->p.u_stride = stride;
    for (int i = 0; i < 3; ++i) c->p.split[i] = (int32_t)s.channels[i];
    c->p.width = (int32_t)(c->width > 1000 ? 1000 : c->width);
    c->p.nseq = (int32_t)nseq;
    c->p.dtype = code(u, "u");
    c->p.wdtype = wcode;
    c->p.activation = silu;
}
void three_dims(const Tensor& u) {
    on_gpu(u, "u");
    if (u.dim() != 3) value_error("u must be [batch, L, channels]");
    if (u.size(2) > (1 << 24)) throw Status{SSD_ERR_UNSUPPORTED, "ssd_conv"};
}

// u, weight, bias, split, silu, cu_seqlens, positions, initial_state, final_state, out,
// final_state_out
PyObject* conv_forward(PyObject* const* a) {
    const Tensor& u = tensor(a[0], "u");
    three_dims(u);
    const Tensor& w = tensor(a[1], "weight");
    const Tensor *b = maybe(a[2], "bias"), *cu = maybe(a[5], "cu_seqlens");
    const Tensor *pos = maybe(a[6], "positions"), *init = maybe(a[7], "initial_state");
    const int64_t batch = u.size(0), L = u.size(1), C = u.size(2);
    const auto dev = u.device();
    const auto type = u.scalar_type();
    Pieces s;
    if (a[3] == Py_None) {
        s.add(batch, L);
        if (C > 0) s.dim(C);
    } else {
        PyObject* seq = PySequence_Fast(a[3], "split must be a sequence");
        if (!seq) throw Raised();
        struct Drop {
            PyObject* o;
            ~Drop() { Py_DECREF(o); }
        } drop{seq};
        for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq); ++i) {
            PyObject* e = PySequence_Fast_GET_ITEM(seq, i);
            s.add(batch, L);
            if (PyLong_Check(e)) {
                s.dim(integer(e));
                continue;
            }
            PyObject* inner = PySequence_Fast(e, "split holds sizes or shapes");
            if (!inner) throw Raised();
            Drop drop2{inner};
            for (Py_ssize_t k = 0; k < PySequence_Fast_GET_SIZE(inner); ++k)
                s.dim(integer(PySequence_Fast_GET_ITEM(inner, k)));
        }
        if (s.n == 0) value_error("split must name one to three pieces");
    }
    s.total(C);
    ConvCall c;
    conv_problem(&c, u, w, b, s, truth(a[4]), cu, pos, init);

    const c10::cuda::CUDAGuard guard(dev);
    Tensor o[3], final;
    if (a[9] == Py_None) {
        for (int i = 0; i < s.n; ++i) o[i] = empty(s.shape[i], type, dev);
    } else {
        if (a[3] != Py_None) {
            if (!PyTuple_Check(a[9]) && !PyList_Check(a[9])) type_error("out must be a tuple");
            if (PySequence_Size(a[9]) != s.n)
                value_error("out must hold " + std::to_string(s.n) + " tensors");
        }
        for (int i = 0; i < s.n; ++i) {
            PyObject* e = a[3] == Py_None     ? a[9]
                          : PyTuple_Check(a[9]) ? PyTuple_GET_ITEM(a[9], i)
                                                : PyList_GET_ITEM(a[9], i);
            o[i] = tensor(e, "out");
            check(o[i], "out", dev, type, s.shape[i]);
        }
    }
    if (a[10] != Py_None) {
        final = tensor(a[10], "final_state_out");
        check(final, "final_state_out", dev, type, {c.n, c.width, C});
    } else if (truth(a[8])) {
        final = empty({c.n, c.width, C}, type, dev);
    }
    void* op[3] = {nullptr, nullptr, nullptr};
    for (int i = 0; i < s.n; ++i) op[i] = o[i].data_ptr();
    ok(ssd_conv_forward(&c.p, u.data_ptr(), w.data_ptr(), ptr(b), static_cast<int32_t*>(ptr(cu)),
                        static_cast<int32_t*>(ptr(pos)), ptr(init), op[0], op[1], op[2],
                        final.defined() ? final.data_ptr() : nullptr, stream_of(dev)),
       "ssd_conv_forward");
    PyObject* outs;
    if (a[3] == Py_None)
        outs = wrap(o[0]);
    else if (s.n == 1)
        outs = tuple({wrap(o[0])});
    else if (s.n == 2)
        outs = tuple({wrap(o[0]), wrap(o[1])});
    else
        outs = tuple({wrap(o[0]), wrap(o[1]), wrap(o[2])});
    return tuple({outs, wrap(final)});
}

// u, weight, bias, dy, silu, cu_seqlens, positions, initial_state, d_final_state,
// d_initial_state, out, workspace
PyObject* conv_backward(PyObject* const* a) {
    const Tensor& u = tensor(a[0], "u");
    three_dims(u);
    const Tensor& w = tensor(a[1], "weight");
    const Tensor *b = maybe(a[2], "bias"), *cu = maybe(a[5], "cu_seqlens");
    const Tensor *pos = maybe(a[6], "positions"), *init = maybe(a[7], "initial_state");
    const Tensor* dfinal = maybe(a[8], "d_final_state");
    const int64_t batch = u.size(0), L = u.size(1), C = u.size(2);
    const auto dev = u.device();
    const auto type = u.scalar_type();
    Pieces s;
    const void* dp[3] = {nullptr, nullptr, nullptr};
    const bool one = THPVariable_Check(a[3]);
    if (!one && !PyTuple_Check(a[3]) && !PyList_Check(a[3]))
        type_error("dy must be a tensor or a tuple of tensors");
    const Py_ssize_t nd = one ? 1 : PySequence_Size(a[3]);
    if (nd < 1 || nd > 3) value_error("dy must be one to three tensors");
    for (Py_ssize_t i = 0; i < nd; ++i) {
        PyObject* e = one                   ? a[3]
                      : PyTuple_Check(a[3]) ? PyTuple_GET_ITEM(a[3], i)
                                            : PyList_GET_ITEM(a[3], i);
        const Tensor& d = tensor(e, "dy");
        if (d.dim() < 3 || d.size(0) != batch || d.size(1) != L)
            value_error("dy must be [batch, L, ...]");
        on_device(d, "dy", dev);
        of_type(d, "dy", type);
        contiguous(d, "dy");
        s.add(batch, L);
        for (int64_t k = 2; k < d.dim(); ++k) s.dim(d.size(k));
        dp[i] = d.data_ptr();
    }
    s.total(C);
    ConvCall c;
    conv_problem(&c, u, w, b, s, truth(a[4]), cu, pos, init);
    if (dfinal) check(*dfinal, "d_final_state", dev, type, {c.n, c.width, C});

    const c10::cuda::CUDAGuard guard(dev);
    Dict g(a[10]);
    Tensor du = brought(a[10], "du"), dw = brought(a[10], "d_weight"), db, d0;
    if (du.defined())
        c.p.du_stride = rows(du, "du", dev, type, u.sizes());
    else
        du = empty(u.sizes(), type, dev), c.p.du_stride = C;
    if (dw.defined())
        check(dw, "d_weight", dev, w.scalar_type(), w.sizes());
    else
        dw = empty(w.sizes(), w.scalar_type(), dev);
    // what `out` brings is written (or refused), asked for by its argument or not
    db = brought(a[10], "d_bias");
    if (db.defined()) {
        if (!b) value_error("out brings d_bias, but there is no bias");
        check(db, "d_bias", dev, w.scalar_type(), {C});
    } else if (b) {
        db = empty({C}, w.scalar_type(), dev);
    }
    d0 = brought(a[10], "d_initial_state");
    if (d0.defined())
        check(d0, "d_initial_state", dev, type, {c.n, c.width, C});
    else if (truth(a[9]))
        d0 = empty({c.n, c.width, C}, type, dev);
    size_t need = 0;
    ok(ssd_conv_workspace_size(&c.p, &need), "ssd_conv_workspace_size");
    const Scratch ws(a[11], need, dev);
    ok(ssd_conv_backward(&c.p, u.data_ptr(), w.data_ptr(), ptr(b), static_cast<int32_t*>(ptr(cu)),
                         static_cast<int32_t*>(ptr(pos)), ptr(init), dp[0], dp[1], dp[2], ptr(dfinal),
                         du.data_ptr(), dw.data_ptr(), db.defined() ? db.data_ptr() : nullptr,
                         d0.defined() ? d0.data_ptr() : nullptr, ws.p, ws.n, stream_of(dev)),
       "ssd_conv_backward");
    g.set("du", du);
    g.set("d_weight", dw);
    if (db.defined()) g.set("d_bias", db);
    if (d0.defined()) g.set("d_initial_state", d0);
    return g.release();
}

// state, conv_state, u, raw_dt, weight, bias, positions, delta_init, ngroups, slots, out
PyObject* conv_decode_step(PyObject* const* a) {
    const Tensor &state = tensor(a[0], "state"), &win = tensor(a[1], "conv_state");
    const Tensor &u = tensor(a[2], "u"), &raw = tensor(a[3], "raw_dt");
    const Tensor& w = tensor(a[4], "weight");
    const Tensor *b = maybe(a[5], "bias"), *slots = maybe(a[9], "slots");
    const Tensor& pos = tensor(a[6], "positions");
    on_gpu(u, "u");
    if (u.dim() != 2 || state.dim() != 4)
        value_error("u must be [batch, channels], state [nslots, H, P, N]");
    const auto dev = u.device();
    const auto type = u.scalar_type();
    const int64_t stride = rows(u, "u"), batch = u.size(0), C = u.size(1);
    const int64_t n = state.size(0), H = state.size(1), P = state.size(2), N = state.size(3);
    const int32_t G = int32(a[8], "ngroups");
    if (C != H * P + 2 * G * N)
        value_error("u has " + std::to_string(C) + " channels, H P + 2 ngroups N is " +
                    std::to_string(H * P + 2 * G * N));
    if (w.dim() != 2 || w.size(0) != C) value_error("weight must be [channels, width]");
    if (n > INT32_MAX || batch > INT32_MAX || C > (1 << 24))
        throw Status{SSD_ERR_UNSUPPORTED, "ssd_conv_decode_step"};
    const int64_t width = w.size(1);
    on_device(w, "weight", dev);
    contiguous(w, "weight");
    const int wcode = code(w, "weight");
    if (b) check(*b, "bias", dev, w.scalar_type(), {C});
    on_device(state, "state", dev);
    of_type(state, "state", at::kFloat);
    contiguous(state, "state");
    check(win, "conv_state", dev, type, {n, width, C});
    check(raw, "raw_dt", dev, at::kFloat, {batch, H});
    check(pos, "positions", dev, at::kInt, {batch});
    if (slots) check(*slots, "slots", dev, at::kInt, {batch});
    ssd_problem_t p = {};
    p.batch = batch, p.seqlen = 1;
    p.nheads = (int32_t)H, p.headdim = (int32_t)P, p.dstate = (int32_t)N, p.ngroups = G;
    p.chunk_size = 64;
    p.delta_init = (float)number(a[7]);
    p.dtype = code(u, "u");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor y;
    if (a[10] == Py_None) {
        y = empty({batch, H, P}, type, dev);
    } else {
        y = tensor(a[10], "out");
        check(y, "out", dev, type, {batch, H, P});
    }
    ok(ssd_conv_decode_step(&p, (int32_t)(width > 1000 ? 1000 : width), wcode, (int32_t)n, stride,
                            static_cast<float*>(state.data_ptr()), win.data_ptr(), u.data_ptr(),
                            static_cast<float*>(raw.data_ptr()), w.data_ptr(), ptr(b),
                            static_cast<int32_t*>(pos.data_ptr()), static_cast<int32_t*>(ptr(slots)),
                            y.data_ptr(), stream_of(dev)),
       "ssd_conv_decode_step");
    return wrap(y);
}

// ------------------------------------------------------------------ norms
int64_t columns(const Tensor& t, const char* name) {
    const int64_t D = t.size(-1);
    if (D < 1 || D > INT32_MAX) value_error(std::string(name) + " must have columns");
    return D;
}
int weight_of(const Tensor& w, const Tensor* b, at::Device dev, int64_t D) {
    const int c = code(w, "weight");
    check(w, "weight", dev, w.scalar_type(), {D});
    if (b) check(*b, "bias", dev, w.scalar_type(), {D});
    return c;
}

// x, weight, bias, residual, eps, kind, out, residual_out, stats
PyObject* norm_forward(PyObject* const* a) {
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
    const Tensor *b = maybe(a[2], "bias"), *res = maybe(a[3], "residual");
    on_gpu(x, "x");
    const auto dev = x.device();
    const auto type = x.scalar_type();
    ssd_norm_t p = {};
    p.x_stride = rows(x, "x");
    const int64_t D = columns(x, "x");
    p.rows = x.numel() / D;
    p.dim = (int32_t)D;
    p.dtype = code(x, "x");
    p.wdtype = weight_of(w, b, dev, D);
    p.kind = int32(a[5], "kind");
    p.eps = (float)number(a[4]);
    p.r_stride = p.h_stride = p.y_stride = D;
    p.rdtype = p.dtype;
    auto rtype = type;
    if (res) {
        rtype = res->scalar_type();
        p.rdtype = code(*res, "residual");
        p.r_stride = rows(*res, "residual", dev, rtype, x.sizes());
    }
    const c10::cuda::CUDAGuard guard(dev);
    Tensor y, h, stats;
    if (a[6] == Py_None) {
        y = empty(x.sizes(), type, dev);
    } else {
        y = tensor(a[6], "out");
        p.y_stride = rows(y, "out", dev, type, x.sizes());
    }
    if (res) {
        if (a[7] == Py_None) {
            h = empty(x.sizes(), rtype, dev);
        } else {
            h = tensor(a[7], "residual_out");
            p.h_stride = rows(h, "residual_out", dev, rtype, x.sizes());
        }
    } else if (a[7] != Py_None) {
        value_error("residual_out without a residual: h is x itself");
    }
    if (truth(a[8])) stats = empty({p.rows, 2}, at::kFloat, dev);
    ok(ssd_norm_forward(&p, x.data_ptr(), ptr(res), w.data_ptr(), ptr(b), y.data_ptr(),
                        res ? h.data_ptr() : nullptr,
                        stats.defined() ? static_cast<float*>(stats.data_ptr()) : nullptr,
                        stream_of(dev)),
       "ssd_norm_forward");
    PyObject* ho = a[0];
    if (res)
        ho = wrap(h);
    else
        Py_INCREF(ho);
    return tuple({wrap(y), ho, wrap(stats)});
}

// dy, h, weight, stats, dh, kind, bias, out, workspace
PyObject* norm_backward(PyObject* const* a) {
    const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h"), &w = tensor(a[2], "weight");
    const Tensor& stats = tensor(a[3], "stats");
    const Tensor* dh = maybe(a[4], "dh");
    on_gpu(dy, "dy");
    const auto dev = dy.device();
    const auto type = dy.scalar_type(), rtype = h.scalar_type();
    ssd_norm_t p = {};
    p.y_stride = rows(dy, "dy");
    const int64_t D = columns(dy, "dy");
    p.rows = dy.numel() / D;
    p.dim = (int32_t)D;
    p.dtype = code(dy, "dy");
    p.rdtype = code(h, "h");
    p.h_stride = rows(h, "h", dev, rtype, dy.sizes());
    p.wdtype = weight_of(w, nullptr, dev, D);
    p.kind = int32(a[5], "kind");
    check(stats, "stats", dev, at::kFloat, {p.rows, 2});
    p.r_stride = dh ? rows(*dh, "dh", dev, rtype, dy.sizes()) : D;
    const c10::cuda::CUDAGuard guard(dev);
    Dict g(a[7]);
    Tensor dx = brought(a[7], "dx"), dw = brought(a[7], "d_weight"), db, dres;
    if (dx.defined())
        p.x_stride = rows(dx, "dx", dev, type, dy.sizes());
    else
        dx = empty(dy.sizes(), type, dev), p.x_stride = D;
    // d_residual is dx itself where the types agree, unless `out` brings another tensor for it
    // (an earlier call's dict brings dx again)
    dres = brought(a[7], "d_residual");
    const bool again = dres.defined() && dres.scalar_type() == type && rtype == type &&
                       dres.data_ptr() == dx.data_ptr() && dres.sizes() == dx.sizes() &&
                       dres.strides() == dx.strides();
    if (again)
        dres = Tensor();
    else if (dres.defined())
        check(dres, "d_residual", dev, rtype, dy.sizes());
    else if (rtype != type)
        dres = empty(dy.sizes(), rtype, dev);
    if (dw.defined())
        check(dw, "d_weight", dev, w.scalar_type(), {D});
    else
        dw = empty({D}, w.scalar_type(), dev);
    db = brought(a[7], "d_bias");  // what `out` brings is written, asked for or not
    if (db.defined())
        check(db, "d_bias", dev, w.scalar_type(), {D});
    else if (truth(a[6]))
        db = empty({D}, w.scalar_type(), dev);
    size_t need = 0;
    ok(ssd_norm_workspace_size(&p, &need), "ssd_norm_workspace_size");
    const Scratch ws(a[8], need, dev);
    ok(ssd_norm_backward(&p, dy.data_ptr(), h.data_ptr(), ptr(dh), w.data_ptr(),
                         static_cast<float*>(stats.data_ptr()), dx.data_ptr(),
                         dres.defined() ? dres.data_ptr() : nullptr, dw.data_ptr(),
                         db.defined() ? db.data_ptr() : nullptr, ws.p, ws.n, stream_of(dev)),
       "ssd_norm_backward");
    g.set("dx", dx);
    if (dres.defined()) {
        g.set("d_residual", dres);
    } else if (dh && !again) {
        PyObject* same = PyDict_GetItemString(g.d, "dx");
        if (PyDict_SetItemString(g.d, "d_residual", same) < 0) throw Raised();
    }
    g.set("d_weight", dw);
    if (db.defined()) g.set("d_bias", db);
    return g.release();
}

// The row stride of y: of z's shape, or contiguous with z's last dimension split in two.
int64_t like_gate(const Tensor& y, const char* name, const Tensor& z) {
    on_device(y, name, z.device());
    of_type(y, name, z.scalar_type());
    if (y.sizes() == z.sizes()) return rows(y, name);
    const int64_t d = z.dim();
    bool fits = y.dim() == d + 1 && y.size(d - 1) * y.size(d) == z.size(d - 1);
    for (int64_t i = 0; fits && i < d - 1; ++i) fits = y.size(i) == z.size(i);
    if (!fits)
        value_error(std::string(name) + " must be [..., D] as z, or [..., H, P] with H P = D");
    contiguous(y, name);
    return z.size(d - 1);
}

// y, z, weight, eps, groups, out
PyObject* gated_norm_forward(PyObject* const* a) {
    const Tensor &y = tensor(a[0], "y"), &z = tensor(a[1], "z"), &w = tensor(a[2], "weight");
    on_gpu(z, "z");
    const auto dev = z.device();
    ssd_gated_norm_t p = {};
    p.z_stride = rows(z, "z");
    const int64_t D = columns(z, "z");
    p.rows = z.numel() / D;
    p.dim = (int32_t)D;
    p.y_stride = like_gate(y, "y", z);
    p.out_stride = p.dy_stride = p.dz_stride = D;
    p.dtype = code(z, "z");
    p.wdtype = weight_of(w, nullptr, dev, D);
    p.eps = (float)number(a[3]);
    p.groups = int32(a[4], "groups");
    if (p.groups < 1) value_error("groups must be positive");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor o, rstd = empty({p.rows, p.groups}, at::kFloat, dev);
    if (a[5] == Py_None) {
        o = empty(z.sizes(), z.scalar_type(), dev);
    } else {
        o = tensor(a[5], "out");
        p.out_stride = rows(o, "out", dev, z.scalar_type(), z.sizes());
    }
    ok(ssd_gated_norm_forward(&p, y.data_ptr(), z.data_ptr(), w.data_ptr(), o.data_ptr(),
                              static_cast<float*>(rstd.data_ptr()), stream_of(dev)),
       "ssd_gated_norm_forward");
    return tuple({wrap(o), wrap(rstd)});
}

// dout, y, z, weight, rstd, groups, out, workspace
PyObject* gated_norm_backward(PyObject* const* a) {
    const Tensor &dout = tensor(a[0], "dout"), &y = tensor(a[1], "y"), &z = tensor(a[2], "z");
    const Tensor &w = tensor(a[3], "weight"), &rstd = tensor(a[4], "rstd");
    on_gpu(z, "z");
    const auto dev = z.device();
    const auto type = z.scalar_type();
    ssd_gated_norm_t p = {};
    p.z_stride = rows(z, "z");
    const int64_t D = columns(z, "z");
    p.rows = z.numel() / D;
    p.dim = (int32_t)D;
    p.y_stride = like_gate(y, "y", z);
    p.out_stride = rows(dout, "dout", dev, type, z.sizes());
    p.dtype = code(z, "z");
    p.wdtype = weight_of(w, nullptr, dev, D);
    p.groups = int32(a[5], "groups");
    if (p.groups < 1) value_error("groups must be positive");
    check(rstd, "rstd", dev, at::kFloat, {p.rows, p.groups});
    const c10::cuda::CUDAGuard guard(dev);
    Dict g(a[6]);
    Tensor dy = brought(a[6], "dy"), dz = brought(a[6], "dz"), dw = brought(a[6], "d_weight");
    if (dy.defined()) {
        if (dy.sizes() != y.sizes()) value_error("dy must have the shape of y");
    } else {
        dy = empty(y.sizes(), type, dev);
    }
    p.dy_stride = like_gate(dy, "dy", z);
    if (dz.defined())
        p.dz_stride = rows(dz, "dz", dev, type, z.sizes());
    else
        dz = empty(z.sizes(), type, dev), p.dz_stride = D;
    if (dw.defined())
        check(dw, "d_weight", dev, w.scalar_type(), {D});
    else
        dw = empty({D}, w.scalar_type(), dev);
    size_t need = 0;
    ok(ssd_gated_norm_workspace_size(&p, &need), "ssd_gated_norm_workspace_size");
    const Scratch ws(a[7], need, dev);
    ok(ssd_gated_norm_backward(&p, dout.data_ptr(), y.data_ptr(), z.data_ptr(), w.data_ptr(),
                               static_cast<float*>(rstd.data_ptr()), dy.data_ptr(), dz.data_ptr(),
                               dw.data_ptr(), ws.p, ws.n, stream_of(dev)),
       "ssd_gated_norm_backward");
    g.set("dy", dy);
    g.set("dz", dz);
    g.set("d_weight", dw);
    return g.release();
}

// ------------------------------------------------------------------ linear attention
// The stride between the tokens of t [..., heads, channels], whose heads lie next to one another.
int64_t tokens(const Tensor& t, const char* name) {
    const int64_t d = t.dim(), H = t.size(d - 2), D = t.size(d - 1);
    if (t.is_contiguous()) return H * D;
    if ((D > 1 && t.stride(d - 1) != 1) || (H > 1 && t.stride(d - 2) != D))
        value_error(std::string(name) + ": the heads of a token must lie next to one another");
    int64_t step = -1, span = 1;
    for (int64_t i = d - 3; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (step < 0)
            step = t.stride(i);
        else if (t.stride(i) != span * step)
            value_error(std::string(name) + ": tokens must be evenly spaced");
        span *= t.size(i);
    }
    if (step < 0) return H * D;
    if (step < H * D) value_error(std::string(name) + ": tokens overlap");
    return step;
}
int64_t tokens(const Tensor& t, const char* name, at::Device dev, at::ScalarType type,
               at::IntArrayRef shape) {
    on_device(t, name, dev);
    of_type(t, name, type);
    of_shape(t, name, shape);
    return tokens(t, name);
}

struct AttnCall {
    ssd_linattn_t p;
    int64_t n;
};
void attn_problem(AttnCall* c, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& ld,
                  PyObject* scale, const Tensor* cu, const Tensor* init) {
    on_gpu(q, "q");
    if (q.dim() != 4 || k.dim() != 4 || v.dim() != 4)
        value_error("q must be [batch, L, H, N], k [batch, L, G, N], v [batch, L, G, P]");
    const auto dev = q.device();
    const auto type = q.scalar_type();
    const int64_t B = q.size(0), L = q.size(1), H = q.size(2), N = q.size(3), G = k.size(2), P = v.size(3);
    if (H > INT32_MAX || N > INT32_MAX || P > INT32_MAX || G < 1 || H % G != 0)
        value_error("q has " + std::to_string(H) + " heads, k " + std::to_string(G));
    c->p = {};
    c->p.dtype = code(q, "q");
    c->p.q_stride = tokens(q, "q");
    c->p.k_stride = tokens(k, "k", dev, type, {B, L, G, N});
    c->p.v_stride = tokens(v, "v", dev, type, {B, L, G, P});
    check(ld, "log_decay", dev, at::kFloat, {H});
    int64_t nseq = 0;
    if (cu) {
        on_device(*cu, "cu_seqlens", dev);
        of_type(*cu, "cu_seqlens", at::kInt);
        contiguous(*cu, "cu_seqlens");
        if (B != 1) value_error("packed sequences need batch == 1");
        nseq = cu->numel() - 1;
        if (cu->dim() != 1 || nseq < 1) value_error("cu_seqlens must be [nseq + 1]");
        if (nseq > INT32_MAX) throw Status{SSD_ERR_UNSUPPORTED, "ssd_linear_attention"};
    }
    c->n = nseq ? nseq : B;
    if (init) check(*init, "initial_state", dev, at::kFloat, {c->n, H, P, N});
    c->p.batch = B, c->p.seqlen = L, c->p.nseq = (int32_t)nseq;
    c->p.nheads = (int32_t)H, c->p.ngroups = (int32_t)G, c->p.headdim = (int32_t)P, c->p.dstate = (int32_t)N;
    c->p.o_stride = H * P;
    c->p.scale = scale == Py_None ? (float)(1.0 / std::sqrt((double)N)) : (float)number(scale);
}
// Bytes of workspace; where the call brings none, also for the copies by which tensors that do not start
// on 16 bytes reach the tensor cores.
size_t attn_workspace(const ssd_linattn_t& p, int bwd, PyObject* given, std::initializer_list<const Tensor*> tensors) {
    size_t need = 0, more = 0;
    ok(ssd_linear_attention_workspace_size(&p, bwd, &need), "ssd_linear_attention_workspace_size");
    uintptr_t at = 0;
    for (const Tensor* t : tensors) at |= (uintptr_t)t->data_ptr();
    if (given != Py_None || at % 16 == 0) return need;
    ssd_linattn_t odd = p;
    odd.q_stride |= 1;
    ok(ssd_linear_attention_workspace_size(&odd, bwd, &more), "ssd_linear_attention_workspace_size");
    return need > more ? need : more;
}
float* floats(const Tensor* t) { return static_cast<float*>(ptr(t)); }
float* floats(const Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; }
int32_t* ints(const Tensor* t) { return static_cast<int32_t*>(ptr(t)); }

// q, k, v, log_decay, scale, cu_seqlens, initial_state, final_state, out, final_state_out, workspace
PyObject* linear_attention_forward(PyObject* const* a) {
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const Tensor& ld = tensor(a[3], "log_decay");
    const Tensor *cu = maybe(a[5], "cu_seqlens"), *init = maybe(a[6], "initial_state");
    AttnCall c;
    attn_problem(&c, q, k, v, ld, a[4], cu, init);
    const auto dev = q.device();
    const int64_t B = q.size(0), L = q.size(1), H = q.size(2), N = q.size(3), P = v.size(3);
    const c10::cuda::CUDAGuard guard(dev);
    Tensor o, final;
    if (a[8] == Py_None) {
        o = empty({B, L, H, P}, q.scalar_type(), dev);
    } else {
        o = tensor(a[8], "out");
        c.p.o_stride = tokens(o, "out", dev, q.scalar_type(), {B, L, H, P});
    }
    if (a[9] != Py_None) {
        final = tensor(a[9], "final_state_out");
        check(final, "final_state_out", dev, at::kFloat, {c.n, H, P, N});
    } else if (truth(a[7])) {
        final = empty({c.n, H, P, N}, at::kFloat, dev);
    }
    const Scratch ws(a[10], attn_workspace(c.p, 0, a[10], {&q, &k, &v, &o}), dev);
    ok(ssd_linear_attention_forward(&c.p, q.data_ptr(), k.data_ptr(), v.data_ptr(), floats(&ld), ints(cu),
                                    floats(init), o.data_ptr(), floats(final), ws.p, ws.n, stream_of(dev)),
       "ssd_linear_attention_forward");
    return tuple({wrap(o), wrap(final)});
}

// q, k, v, log_decay, do, scale, cu_seqlens, initial_state, d_final_state, d_initial_state, out,
// workspace
PyObject* linear_attention_backward(PyObject* const* a) {
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const Tensor &ld = tensor(a[3], "log_decay"), &dout = tensor(a[4], "do");
    const Tensor *cu = maybe(a[6], "cu_seqlens"), *init = maybe(a[7], "initial_state");
    const Tensor* dfinal = maybe(a[8], "d_final_state");
    AttnCall c;
    attn_problem(&c, q, k, v, ld, a[5], cu, init);
    const auto dev = q.device();
    const auto type = q.scalar_type();
    const int64_t B = q.size(0), L = q.size(1), H = q.size(2), N = q.size(3), P = v.size(3);
    c.p.o_stride = tokens(dout, "do", dev, type, {B, L, H, P});
    if (dfinal) check(*dfinal, "d_final_state", dev, at::kFloat, {c.n, H, P, N});
    const c10::cuda::CUDAGuard guard(dev);
    Dict g(a[10]);
    struct Grad {
        const char* name;
        const Tensor& of;
        int64_t* stride;
        Tensor t;
    } grads[3] = {{"dq", q, &c.p.dq_stride, {}}, {"dk", k, &c.p.dk_stride, {}}, {"dv", v, &c.p.dv_stride, {}}};
    for (Grad& d : grads) {
        d.t = brought(a[10], d.name);
        if (d.t.defined())
            *d.stride = tokens(d.t, d.name, dev, type, d.of.sizes());
        else
            d.t = empty(d.of.sizes(), type, dev), *d.stride = d.of.size(2) * d.of.size(3);
    }
    Tensor d0 = brought(a[10], "d_initial_state");  // what `out` brings is written, asked for or not
    if (d0.defined())
        check(d0, "d_initial_state", dev, at::kFloat, {c.n, H, P, N});
    else if (truth(a[9]))
        d0 = empty({c.n, H, P, N}, at::kFloat, dev);
    const Scratch ws(a[11], attn_workspace(c.p, 1, a[11], {&q, &k, &v, &dout, &grads[0].t, &grads[1].t, &grads[2].t}),
                     dev);
    ok(ssd_linear_attention_backward(&c.p, q.data_ptr(), k.data_ptr(), v.data_ptr(), floats(&ld), ints(cu),
                                     floats(init), dout.data_ptr(), floats(dfinal), grads[0].t.data_ptr(),
                                     grads[1].t.data_ptr(), grads[2].t.data_ptr(), floats(d0), ws.p, ws.n,
                                     stream_of(dev)),
       "ssd_linear_attention_backward");
    for (const Grad& d : grads) g.set(d.name, d.t);
    if (d0.defined()) g.set("d_initial_state", d0);
    return g.release();
}

// state, q, k, v, log_decay, scale, slots, out
PyObject* linear_attention_step(PyObject* const* a) {
    const Tensor &state = tensor(a[0], "state"), &q = tensor(a[1], "q"), &k = tensor(a[2], "k");
    const Tensor &v = tensor(a[3], "v"), &ld = tensor(a[4], "log_decay");
    const Tensor* slots = maybe(a[6], "slots");
    on_gpu(q, "q");
    if (q.dim() != 3 || k.dim() != 3 || v.dim() != 3 || state.dim() != 4)
        value_error("q must be [batch, H, N], k [batch, G, N], v [batch, G, P], state [nslots, H, P, N]");
    const auto dev = q.device();
    const auto type = q.scalar_type();
    const int64_t B = q.size(0), H = q.size(1), N = q.size(2), G = k.size(1), P = v.size(2), n = state.size(0);
    if (G < 1 || H % G != 0)
        value_error("q has " + std::to_string(H) + " heads, k " + std::to_string(G));
    if (n > INT32_MAX || H > INT32_MAX || N > INT32_MAX || P > INT32_MAX)
        throw Status{SSD_ERR_UNSUPPORTED, "ssd_linear_attention_step"};
    ssd_linattn_t p = {};
    p.batch = B, p.seqlen = 1;
    p.nheads = (int32_t)H, p.ngroups = (int32_t)G, p.headdim = (int32_t)P, p.dstate = (int32_t)N;
    p.dtype = code(q, "q");
    p.q_stride = tokens(q, "q");
    p.k_stride = tokens(k, "k", dev, type, {B, G, N});
    p.v_stride = tokens(v, "v", dev, type, {B, G, P});
    p.o_stride = H * P;
    p.scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)N)) : (float)number(a[5]);
    check(state, "state", dev, at::kFloat, {n, H, P, N});
    check(ld, "log_decay", dev, at::kFloat, {H});
    if (slots) check(*slots, "slots", dev, at::kInt, {B});
    const c10::cuda::CUDAGuard guard(dev);
    Tensor o;
    if (a[7] == Py_None) {
        o = empty({B, H, P}, type, dev);
    } else {
        o = tensor(a[7], "out");
        p.o_stride = tokens(o, "out", dev, type, {B, H, P});
    }
    ok(ssd_linear_attention_step(&p, (int32_t)n, floats(&state), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                 floats(&ld), ints(slots), o.data_ptr(), stream_of(dev)),
       "ssd_linear_attention_step");
    return wrap(o);
}

// ------------------------------------------------------------------ beam search
// logits, scores, keep, finished, pad_token, out, workspace
PyObject* beam_select(PyObject* const* a) {
    const Tensor &x = tensor(a[0], "logits"), &scores = tensor(a[1], "scores");
    const Tensor* finished = maybe(a[3], "finished");
    on_gpu(x, "logits");
    if (x.dim() != 3) value_error("logits must be [batch, beams, vocab]");
    const auto dev = x.device();
    const int64_t B = x.size(0), K = x.size(1), V = x.size(2);
    if (K > INT32_MAX || V > INT32_MAX) throw Status{SSD_ERR_UNSUPPORTED, "ssd_beam_select"};
    ssd_beam_t p = {};
    p.stride = rows(x, "logits");
    p.dtype = code(x, "logits");
    p.batch = B, p.beams = (int32_t)K, p.vocab = (int32_t)V;
    p.keep = a[2] == Py_None ? p.beams : int32(a[2], "keep");
    p.pad_token = int32(a[4], "pad_token");
    check(scores, "scores", dev, at::kFloat, {B, K});
    if (finished) {
        if (finished->scalar_type() != at::kBool && finished->scalar_type() != at::kByte)
            type_error("finished must be torch.bool or torch.uint8, got " + text(finished->scalar_type()));
        check(*finished, "finished", dev, finished->scalar_type(), {B, K});
    }
    size_t need = 0;
    const c10::cuda::CUDAGuard guard(dev);
    ok(ssd_beam_select_workspace_size(&p, &need), "ssd_beam_select_workspace_size");
    Tensor out[3];
    const at::ScalarType types[3] = {at::kFloat, at::kInt, at::kInt};
    if (a[5] == Py_None) {
        for (int i = 0; i < 3; ++i) out[i] = empty({B, p.keep}, types[i], dev);
    } else {
        if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 3)
            type_error("out must be a tuple (scores, parents, tokens)");
        for (int i = 0; i < 3; ++i) {
            out[i] = tensor(PyTuple_GET_ITEM(a[5], i), "out");
            check(out[i], "out", dev, types[i], {B, p.keep});
        }
    }
    const Scratch ws(a[6], need, dev);
    ok(ssd_beam_select(&p, x.data_ptr(), floats(&scores), static_cast<uint8_t*>(ptr(finished)),
                       floats(out[0]), ints(&out[1]), ints(&out[2]), ws.p, ws.n, stream_of(dev)),
       "ssd_beam_select");
    return tuple({wrap(out[0]), wrap(out[1]), wrap(out[2])});
}

// caches, slots, parents, out
PyObject* beam_reorder(PyObject* const* a) {
    const Tensor &slots = tensor(a[1], "slots"), &parents = tensor(a[2], "parents");
    on_gpu(slots, "slots");
    if (slots.dim() != 2) value_error("slots must be [batch, beams]");
    const auto dev = slots.device();
    const int64_t B = slots.size(0), K = slots.size(1);
    if (K > INT32_MAX) throw Status{SSD_ERR_UNSUPPORTED, "ssd_beam_reorder"};
    check(slots, "slots", dev, at::kInt, {B, K});
    check(parents, "parents", dev, at::kInt, {B, K});
    if (!PyTuple_Check(a[0]) && !PyList_Check(a[0])) type_error("caches must be a list of tensors");
    const Py_ssize_t n = PySequence_Size(a[0]);
    c10::SmallVector<void*, 128> at_;
    c10::SmallVector<int64_t, 128> bytes, strides;
    int64_t nslots = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const Tensor& t = tensor(PyList_Check(a[0]) ? PyList_GET_ITEM(a[0], i) : PyTuple_GET_ITEM(a[0], i), "caches");
        on_device(t, "caches", dev);
        if (t.dim() < 1) value_error("caches must be [nslots, ...]");
        if (nslots >= 0 && t.size(0) != nslots)
            value_error("caches must have the same slots, got " + std::to_string(nslots) + " and " +
                        std::to_string(t.size(0)));
        nslots = t.size(0);
        int64_t span = 1;
        for (int64_t d = t.dim() - 1; d > 0; --d) {
            if (t.size(d) != 1 && t.stride(d) != span) value_error("caches: a slot must be contiguous");
            span *= t.size(d);
        }
        if (nslots > 1 && t.stride(0) < span) value_error("caches: slots overlap");
        if (span == 0) continue;
        const int64_t e = (int64_t)t.element_size();
        at_.push_back(t.data_ptr());
        bytes.push_back(span * e);
        strides.push_back((nslots > 1 ? t.stride(0) : span) * e);
    }
    if (n == 0) nslots = INT32_MAX;
    if (nslots < 1 || nslots > INT32_MAX || at_.size() > INT32_MAX)
        throw Status{nslots < 1 ? SSD_ERR_INVALID_ARG : SSD_ERR_UNSUPPORTED, "ssd_beam_reorder"};
    const c10::cuda::CUDAGuard guard(dev);
    Tensor out;
    if (a[3] == Py_None) {
        out = empty({B, K}, at::kInt, dev);
    } else {
        out = tensor(a[3], "out");
        check(out, "out", dev, at::kInt, {B, K});
    }
    ok(ssd_beam_reorder(B, (int32_t)K, ints(&slots), ints(&parents), ints(&out), (int32_t)at_.size(),
                        at_.data(), bytes.data(), strides.data(), (int32_t)nslots, stream_of(dev)),
       "ssd_beam_reorder");
    return wrap(out);
}

// ------------------------------------------------------------------ module
// No C++ exception leaves a call: ours become Python errors, torch's a RuntimeError.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Err& e) {
        PyErr_SetString(e.type, e.text.c_str());
    } catch (const Status& s) {
        PyObject* o = g_error ? PyObject_CallFunction(g_error, "is", s.code, s.where) : nullptr;
        if (o) {
            PyErr_SetObject(g_error, o);
            Py_DECREF(o);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, ssd_status_string((ssd_status_t)s.code));
        }
    } catch (const Raised&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* m = PyImport_ImportModule("torch");
        PyObject* t = m ? PyObject_GetAttrString(m, "OutOfMemoryError") : nullptr;
        PyErr_Clear();
        PyErr_SetString(t ? t : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(t);
        Py_XDECREF(m);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_XDECREF(g_error);
    Py_INCREF(type);
    g_error = type;
    Py_RETURN_NONE;
}

#define ENTRY(name, n)                                                                     \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), \
     METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(conv_forward, 11),
                         ENTRY(conv_backward, 12),
                         ENTRY(conv_decode_step, 11),
                         ENTRY(norm_forward, 9),
                         ENTRY(norm_backward, 9),
                         ENTRY(gated_norm_forward, 6),
                         ENTRY(gated_norm_backward, 8),
                         ENTRY(linear_attention_forward, 11),
                         ENTRY(linear_attention_backward, 12),
                         ENTRY(linear_attention_step, 8),
                         ENTRY(beam_select, 7),
                         ENTRY(beam_reorder, 4),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_ext", nullptr, -1, methods,
                      nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_ext(void) { return PyModule_Create(&module); }
