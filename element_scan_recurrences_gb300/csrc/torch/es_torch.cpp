// es_torch.cpp -- the sequence-layer operators' marshalling for PyTorch tensors
// (module es_torch, linked to libes.so): checks tensors, fills the argument
// structs of es.h, allocates what the caller did not pass, calls the C ABI on
// the stream.  The same steps in Python cost 12 to 30 us a call on the host,
// which is all of a small call's time; here they are about 1 us.  No
// computation happens here.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "es.h"

namespace {

PyObject* g_es_error = nullptr;      // binding.EsError(status, message)

struct Refused {
    int status;                      // 0: a TypeError
    std::string what;
};

// A Python exception is set already.
struct Raised {};

[[noreturn]] void refuse(int status, const std::string& what) { throw Refused{status, what}; }
[[noreturn]] void wrong_type(const std::string& what) { throw Refused{0, what}; }

PyObject* raise(const Refused& r) {
    if (r.status == 0) {
        PyErr_SetString(PyExc_TypeError, r.what.c_str());
    } else {
        PyObject* e = PyObject_CallFunction(g_es_error, "is", r.status, r.what.c_str());
        if (e != nullptr) {
            PyErr_SetObject(g_es_error, e);
            Py_DECREF(e);
        }
    }
    return nullptr;
}

void check(es_status st) {
    if (st != ES_OK) refuse(st, es_last_error());
}

std::string shape_of(at::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

// A tensor argument; nullopt for None.
std::optional<at::Tensor> maybe(PyObject* o, const char* name) {
    if (o == nullptr || o == Py_None) return std::nullopt;
    if (!THPVariable_Check(o)) wrong_type(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

at::Tensor tensor(PyObject* o, const char* name) {
    auto t = maybe(o, name);
    if (!t) wrong_type(std::string(name) + " must be a torch.Tensor");
    return *t;
}

// An argument's truth value, which an object may refuse to have.
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

// The first operand fixes the type and the device.
at::Tensor first(PyObject* o, const char* name) {
    at::Tensor t = tensor(o, name);
    if (!t.is_cuda() || (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16))
        wrong_type(std::string(name) + " must be a float32 or bfloat16 CUDA tensor");
    return t;
}

int64_t dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? ES_BF16 : ES_F32; }

void like(const at::Tensor& t, const char* name, at::ScalarType type, const at::Device& dev) {
    if (t.scalar_type() != type || t.device() != dev)
        wrong_type(std::string(name) + " must be a " + at::toString(type) + " tensor on " + dev.str() + " (got " +
                   at::toString(t.scalar_type()) + " on " + t.device().str() + ")");
}

// [B, T, heads, dim], or [B, heads, dim] for a step
es_heads view(const at::Tensor& t, const char* name, at::ScalarType type, const at::Device& dev, int rank) {
    like(t, name, type, dev);
    if (t.dim() != rank)
        refuse(ES_E_DIM_001, std::string("E-DIM-001 ") + name + " has rank " + std::to_string(t.dim()) + ", not " + std::to_string(rank));
    const auto s = t.strides();
    const auto n = t.sizes();
    if (s[rank - 1] != 1 && n[rank - 1] > 1 && t.numel() > 0)
        refuse(ES_E_ARG, std::string("the last axis of ") + name + " has stride " + std::to_string(s[rank - 1]) + "; it must be 1");
    if (rank == 3) return es_heads{t.data_ptr(), s[0], 0, s[1], n[1]};
    return es_heads{t.data_ptr(), s[0], s[1], s[2], n[2]};
}

void shaped(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
    if (t.sizes() != shape)
        refuse(ES_E_DIM_001, std::string("E-DIM-001 ") + name + " has shape " + shape_of(t.sizes()) + ", not " + shape_of(shape));
}

// a dense tensor of one dtype and shape (null for None)
void* dense(const std::optional<at::Tensor>& t, const char* name, at::ScalarType type, const at::Device& dev, at::IntArrayRef shape) {
    if (!t) return nullptr;
    like(*t, name, type, dev);
    if (!t->is_contiguous()) wrong_type(std::string(name) + " must be contiguous");
    shaped(*t, name, shape);
    return t->data_ptr();
}

at::Tensor empty(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type));
}

// The call's device and stream: the current stream of the operands' device
// unless one is given (a torch.cuda.Stream or a handle).
struct On {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard stream;
    es_stream_t handle;
    On(const at::Device& dev, PyObject* s) {
        if (c10::cuda::current_device() != dev.index()) device.set_device(dev);
        if (s != nullptr && s != Py_None) {
            PyObject* number = s;
            const bool object = !PyLong_Check(s);
            if (object && (number = PyObject_GetAttrString(s, "cuda_stream")) == nullptr) {
                PyErr_Clear();
                wrong_type("stream must be a torch.cuda.Stream or a handle");
            }
            const size_t raw = PyLong_AsSize_t(number);
            if (object) Py_DECREF(number);
            if (PyErr_Occurred()) {
                PyErr_Clear();
                wrong_type("stream must be a torch.cuda.Stream or a handle");
            }
            stream.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(raw), dev.index()));
        }
        handle = reinterpret_cast<es_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    }
};

PyObject* wrap(const std::optional<at::Tensor>& t) {
    if (!t) Py_RETURN_NONE;
    return THPVariable_Wrap(*t);
}

PyObject* result(std::initializer_list<std::optional<at::Tensor>> ts) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (r == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const auto& t : ts) {
        PyObject* o = wrap(t);
        if (o == nullptr) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// The operands every form of linear attention shares.
struct Operands {
    at::Tensor q, k, v;
    std::optional<at::Tensor> g;
    at::Device dev{at::kCPU};
    at::ScalarType type;
    es_linear_attention_args a{};
    Operands(PyObject* pq, PyObject* pk, PyObject* pv, PyObject* pg, PyObject* scale, bool step)
        : q(first(pq, "q")), k(tensor(pk, "k")), v(tensor(pv, "v")), g(maybe(pg, "log_decay")), dev(q.device()), type(q.scalar_type()) {
        const int rank = step ? 3 : 4;
        a.dtype = dtype_of(q);
        a.q = view(q, "q", type, dev, rank);
        a.k = view(k, "k", type, dev, rank);
        a.v = view(v, "v", type, dev, rank);
        a.batch = q.size(0);
        a.length = step ? 1 : q.size(1);
        a.key_dim = q.size(rank - 1);
        a.value_dim = v.size(rank - 1);
        if (k.size(0) != a.batch || v.size(0) != a.batch || k.size(rank - 1) != a.key_dim ||
            (!step && (k.size(1) != a.length || v.size(1) != a.length)))
            refuse(ES_E_DIM_001, "E-DIM-001 q " + shape_of(q.sizes()) + ", k " + shape_of(k.sizes()) + " and v " + shape_of(v.sizes()) +
                                     " do not fit");
        a.heads = std::max(a.q.heads, std::max(a.k.heads, a.v.heads));
        if (g) {
            like(*g, "log_decay", at::kFloat, dev);
            const auto s = g->strides();
            a.log_decay = static_cast<const float*>(g->data_ptr());
            if (g->dim() == 1) {
                a.heads = g->size(0);
                a.decay_h = s[0];
                a.decay_per_head = 1;
            } else if (g->dim() == rank - 1 && g->size(0) == a.batch && (step || g->size(1) == a.length)) {
                a.heads = g->size(rank - 2);
                a.decay_b = s[0];
                a.decay_t = step ? 0 : s[1];
                a.decay_h = s[rank - 2];
            } else {
                refuse(ES_E_DIM_001, "E-DIM-001 log_decay " + shape_of(g->sizes()) + " fits neither q " + shape_of(q.sizes()) +
                                         " nor one value a head");
            }
        }
        a.scale = 1.0 / std::sqrt(static_cast<double>(a.key_dim));
        if (scale != Py_None) {
            a.scale = PyFloat_AsDouble(scale);
            if (PyErr_Occurred()) {
                PyErr_Clear();
                wrong_type("scale must be a number");
            }
        }
    }
    std::array<int64_t, 4> state_shape() const { return {a.batch, a.heads, a.key_dim, a.value_dim}; }
};

// A workspace of `bytes`: the caller's, or a new one (null where none is needed).
std::optional<at::Tensor> workspace(PyObject* given, size_t bytes, const at::Tensor& q, void** p, int64_t* n) {
    auto w = maybe(given, "workspace");
    if (!w && bytes > 0) w = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
    if (w) {
        if (w->device() != q.device() || !w->is_contiguous()) wrong_type("workspace must be a contiguous tensor on " + q.device().str());
        *p = w->data_ptr();
        *n = static_cast<int64_t>(w->numel() * w->element_size());
    }
    return w;
}

// q, k, v, log_decay, initial_state, lengths, scale, final_state, out, workspace, stream
PyObject* attention(PyObject* const* x) {
    Operands o(x[0], x[1], x[2], x[3], x[6], false);
    On on(o.dev, x[10]);
    auto& a = o.a;
    const auto shape = o.state_shape();
    const auto init = maybe(x[4], "initial_state"), lengths = maybe(x[5], "lengths");
    a.initial_state = static_cast<const float*>(dense(init, "initial_state", at::kFloat, o.dev, shape));
    a.lengths = static_cast<const int32_t*>(dense(lengths, "lengths", at::kInt, o.dev, {a.batch}));
    std::optional<at::Tensor> fin;
    if (THPVariable_Check(x[7])) fin = THPVariable_Unpack(x[7]);
    else if (truth(x[7])) fin = empty(shape, o.q, at::kFloat);
    a.final_state = static_cast<float*>(dense(fin, "final_state", at::kFloat, o.dev, shape));
    auto out = maybe(x[8], "out");
    const std::array<int64_t, 4> want{a.batch, a.length, a.heads, a.value_dim};
    if (!out) out = empty(want, o.q, o.type);
    else shaped(*out, "out", want);
    a.out = view(*out, "out", o.type, o.dev, 4);
    size_t bytes = 0;
    check(es_linear_attention_workspace(&a, nullptr, &bytes));
    const auto ws = workspace(x[9], bytes, o.q, &a.workspace, &a.workspace_bytes);
    check(es_linear_attention(&a, on.handle));
    return result({out, fin});
}

// q, k, v, log_decay, grad_out, initial_state, grad_final_state, lengths, scale, decay_grad, workspace, stream
PyObject* attention_backward(PyObject* const* x) {
    Operands o(x[0], x[1], x[2], x[3], x[8], false);
    On on(o.dev, x[11]);
    auto& a = o.a;
    const auto shape = o.state_shape();
    const auto init = maybe(x[5], "initial_state"), gfin = maybe(x[6], "grad_final_state"), lengths = maybe(x[7], "lengths");
    a.initial_state = static_cast<const float*>(dense(init, "initial_state", at::kFloat, o.dev, shape));
    a.lengths = static_cast<const int32_t*>(dense(lengths, "lengths", at::kInt, o.dev, {a.batch}));
    const at::Tensor go = tensor(x[4], "grad_out");
    es_linear_attention_grads g{};
    g.grad_out = view(go, "grad_out", o.type, o.dev, 4);
    const std::array<int64_t, 4> want{a.batch, a.length, a.heads, a.value_dim};
    shaped(go, "grad_out", want);
    g.grad_final_state = static_cast<const float*>(dense(gfin, "grad_final_state", at::kFloat, o.dev, shape));
    const at::Tensor gq = empty(o.q.sizes(), o.q, o.type), gk = empty(o.k.sizes(), o.q, o.type), gv = empty(o.v.sizes(), o.q, o.type);
    g.grad_q = view(gq, "grad_q", o.type, o.dev, 4);
    g.grad_k = view(gk, "grad_k", o.type, o.dev, 4);
    g.grad_v = view(gv, "grad_v", o.type, o.dev, 4);
    std::optional<at::Tensor> gg, gi;
    if (truth(x[9]) && o.g) {
        gg = empty(o.g->sizes(), o.q, at::kFloat);
        g.grad_log_decay = static_cast<float*>(gg->data_ptr());
    }
    if (init) {
        gi = empty(shape, o.q, at::kFloat);
        g.grad_initial_state = static_cast<float*>(gi->data_ptr());
    }
    size_t bytes = 0;
    check(es_linear_attention_workspace(&a, &g, &bytes));
    const auto ws = workspace(x[10], bytes, o.q, &a.workspace, &a.workspace_bytes);
    check(es_linear_attention_backward(&a, &g, on.handle));
    return result({gq, gk, gv, gg, gi});
}

// q, k, v, log_decay, state, state_out, scale, out, stream
PyObject* attention_step(PyObject* const* x) {
    Operands o(x[0], x[1], x[2], x[3], x[6], true);
    On on(o.dev, x[8]);
    auto& a = o.a;
    const auto shape = o.state_shape();
    const at::Tensor state = tensor(x[4], "state");
    auto state_out = maybe(x[5], "state_out");
    if (!state_out) state_out = state;
    a.initial_state = static_cast<const float*>(dense(state, "state", at::kFloat, o.dev, shape));
    a.final_state = static_cast<float*>(dense(state_out, "state_out", at::kFloat, o.dev, shape));
    auto out = maybe(x[7], "out");
    const std::array<int64_t, 3> want{a.batch, a.heads, a.value_dim};
    if (!out) out = empty(want, o.q, o.type);
    else shaped(*out, "out", want);
    a.out = view(*out, "out", o.type, o.dev, 3);
    check(es_linear_attention_step(&a, on.handle));
    return result({out, state_out});
}

// The operands of the norm and rotation, from x[0..8]: q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours
struct Rotation {
    at::Tensor q;
    std::optional<at::Tensor> k, wq, wk, cos, sin, positions;
    at::Device dev{at::kCPU};
    at::ScalarType type;
    es_qk_norm_rotate_args a{};
    explicit Rotation(PyObject* const* x)
        : q(first(x[0], "q")), k(maybe(x[1], "k")), wq(maybe(x[2], "q_weight")), wk(maybe(x[3], "k_weight")), cos(maybe(x[4], "cos")),
          sin(maybe(x[5], "sin")), positions(maybe(x[6], "positions")), dev(q.device()), type(q.scalar_type()) {
        a.dtype = dtype_of(q);
        a.q = view(q, "q", type, dev, 4);
        a.batch = q.size(0);
        a.length = q.size(1);
        a.dim = q.size(3);
        if (k) {
            a.k = view(*k, "k", type, dev, 4);
            if (k->size(0) != a.batch || k->size(1) != a.length || k->size(3) != a.dim)
                refuse(ES_E_DIM_001, "E-DIM-001 q " + shape_of(q.sizes()) + " and k " + shape_of(k->sizes()) + " do not fit");
        }
        std::optional<at::ScalarType> wtype;
        for (const auto* w : {&wq, &wk})
            if (*w) {
                const auto t = (*w)->scalar_type();
                if ((t != at::kFloat && t != at::kBFloat16) || (wtype && *wtype != t))
                    wrong_type("q_weight and k_weight must be tensors of one dtype, float32 or bfloat16");
                wtype = t;
            }
        a.weight_dtype = wtype && *wtype == at::kBFloat16 ? ES_BF16 : ES_F32;
        a.q_weight = wq ? dense(wq, "q_weight", *wtype, dev, {a.dim}) : nullptr;
        a.k_weight = wk ? dense(wk, "k_weight", *wtype, dev, {a.dim}) : nullptr;
        if (cos) {
            if (cos->dim() != 2) wrong_type("cos must be a [rows, turned / 2] float32 tensor");
            if (!sin) wrong_type("cos without sin");
            a.table_rows = cos->size(0);
            a.turned = 2 * cos->size(1);
            a.cos = static_cast<const float*>(dense(cos, "cos", at::kFloat, dev, cos->sizes()));
            a.sin = static_cast<const float*>(dense(sin, "sin", at::kFloat, dev, cos->sizes()));
        } else if (sin) {
            wrong_type("sin without cos");
        }
        if (positions) {
            const auto t = positions->scalar_type();
            if ((t != at::kInt && t != at::kLong) || positions->device() != dev)
                wrong_type("positions must be an int32 or int64 tensor on " + dev.str());
            a.positions = positions->data_ptr();
            a.positions_64 = t == at::kLong;
            if (positions->dim() == 2 && positions->size(0) == a.batch && positions->size(1) == a.length) {
                a.position_b = positions->stride(0);
                a.position_t = positions->stride(1);
            } else if (positions->dim() == 1 && positions->size(0) == a.length) {
                a.position_t = positions->stride(0);
            } else {
                refuse(ES_E_DIM_001, "E-DIM-001 positions " + shape_of(positions->sizes()) + " fit neither [B, T] nor [T] of q " +
                                         shape_of(q.sizes()));
            }
        }
        a.eps = PyFloat_AsDouble(x[7]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            wrong_type("eps must be a number");
        }
        a.neighbours = truth(x[8]);
    }
    // a result's tensor (a new dense one unless given) and its view
    at::Tensor out(PyObject* given, const at::Tensor& like, const char* name, es_heads* v) {
        auto t = maybe(given, name);
        if (!t) t = empty(like.sizes(), like, type);
        shaped(*t, name, like.sizes());
        *v = view(*t, name, type, dev, 4);
        return *t;
    }
};

// ..., q_out, k_out, stream
PyObject* rotate(PyObject* const* x) {
    Rotation r(x);
    On on(r.dev, x[11]);
    const at::Tensor q = r.out(x[9], r.q, "q_out", &r.a.q_out);
    std::optional<at::Tensor> k;
    if (r.k) k = r.out(x[10], *r.k, "k_out", &r.a.k_out);
    check(es_qk_norm_rotate(&r.a, on.handle));
    return result({q, k});
}

// ..., grad_q_out, grad_k_out, workspace, stream
PyObject* rotate_backward(PyObject* const* x) {
    Rotation r(x);
    On on(r.dev, x[12]);
    es_qk_norm_rotate_grads g{};
    const at::Tensor gqo = tensor(x[9], "grad_q_out");
    g.grad_q_out = view(gqo, "grad_q_out", r.type, r.dev, 4);
    shaped(gqo, "grad_q_out", r.q.sizes());
    std::optional<at::Tensor> gko, gk, gwq, gwk;
    if (r.k) {
        gko = tensor(x[10], "grad_k_out");
        g.grad_k_out = view(*gko, "grad_k_out", r.type, r.dev, 4);
        shaped(*gko, "grad_k_out", r.k->sizes());
    }
    const at::Tensor gq = r.out(Py_None, r.q, "grad_q", &r.a.q_out);
    if (r.k) gk = r.out(Py_None, *r.k, "grad_k", &r.a.k_out);
    if (r.wq) {
        gwq = empty(r.wq->sizes(), *r.wq, r.wq->scalar_type());
        g.grad_q_weight = gwq->data_ptr();
    }
    if (r.wk && r.k) {
        gwk = empty(r.wk->sizes(), *r.wk, r.wk->scalar_type());
        g.grad_k_weight = gwk->data_ptr();
    }
    size_t bytes = 0;
    check(es_qk_norm_rotate_workspace(&r.a, &g, &bytes));
    const auto ws = workspace(x[11], bytes, r.q, &r.a.workspace, &r.a.workspace_bytes);
    check(es_qk_norm_rotate_backward(&r.a, &g, on.handle));
    return result({gq, gk, gwq, gwk});
}

// One Python entry: the number of arguments is fixed (sequence.py passes them
// all), every exception becomes a Python one.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments; %zd are expected", n, N);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& r) {
        return raise(r);
    } catch (const Raised&) {
        return nullptr;
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// the exception class of refusals, set once by sequence.py
PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_es_error);
    g_es_error = cls;
    Py_RETURN_NONE;
}

#define ENTRY(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    ENTRY("linear_attention", attention, 11),
    ENTRY("linear_attention_backward", attention_backward, 12),
    ENTRY("linear_attention_step", attention_step, 9),
    ENTRY("qk_norm_rotate", rotate, 12),
    ENTRY("qk_norm_rotate_backward", rotate_backward, 13),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "es_torch", "Marshalling of PyTorch tensors for libes.so", -1, methods,
                      nullptr,               nullptr,    nullptr,                                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_es_torch() { return PyModule_Create(&module); }
