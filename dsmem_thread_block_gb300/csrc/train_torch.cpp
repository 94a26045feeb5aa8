// train_torch.cpp -- the training operators' calls on torch tensors.
//
// What train.py's functions do between their arguments and the C ABI: check
// the tensors, allocate outputs and workspace from torch's allocator, switch
// to the input's device and take its current stream.  The computation is the C
// ABI's (include/credit.h), reached through function pointers that the binding
// hands over (`bind`), so the checked build can be called the same way.
// Written in C++ because a small call is bound by exactly this work: 20 to 27
// microseconds a call in Python, against a kernel of 2 to 5.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <stdexcept>

#include "credit.h"

namespace {

decltype(&credit_dropout) g_dropout;
decltype(&credit_norm_workspace) g_workspace;
decltype(&credit_norm_forward) g_forward;
decltype(&credit_norm_backward) g_backward;

// A refusal: the Python exception type and its message.
struct Refused {
    PyObject* type;
    const char* message;
};
[[noreturn]] void bad(const char* m) { throw Refused{PyExc_ValueError, m}; }

credit_dtype_t code_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kFloat) return CREDIT_F32;
    if (t.scalar_type() == at::kBFloat16) return CREDIT_BF16;
    throw Refused{PyExc_TypeError, "credit: unsupported dtype (fp32 and bf16 only)"};
}

// An optional tensor argument: None is undefined.
const at::Tensor& tensor(PyObject* o) {
    static const at::Tensor none;
    if (o == Py_None) return none;
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, "credit: a tensor was expected"};
    return THPVariable_Unpack(o);
}

// The calls record no graph: under grad mode a tensor that requires a gradient
// would lose it without a word.
void no_graph(PyObject* const* a, std::initializer_list<int> tensors) {
    if (!c10::GradMode::is_enabled()) return;
    for (const int i : tensors)
        if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).requires_grad())
            throw Refused{PyExc_RuntimeError,
                          "credit: the training operators record no autograd graph, and a tensor "
                          "that requires a gradient was given: call the forward and backward pair "
                          "under torch.no_grad(), or inside a torch.autograd.Function"};
}

// A caller's output has been written: autograd refuses to use what it saved of it.
void written(std::initializer_list<const at::Tensor*> outs) {
    for (const at::Tensor* t : outs)
        if (t->defined() && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The first matrix of a call.
struct Input {
    const at::Tensor& t;
    int64_t rows, cols;
    credit_dtype_t code;
    explicit Input(PyObject* o) : t(tensor(o)) {
        if (!t.defined() || !t.is_cuda() || !t.is_contiguous())
            bad("credit: inputs must be contiguous CUDA tensors");
        if (t.dim() < 1 || t.size(-1) < 1)
            bad("credit: the last dimension must hold at least one element");
        code = code_of(t);
        cols = t.size(-1);
        rows = t.numel() / cols;
    }
    // the pointer of another matrix like it (null: none)
    void* matrix(const at::Tensor& m) const {
        if (!m.defined()) return nullptr;
        if (m.sizes() != t.sizes() || m.scalar_type() != t.scalar_type() ||
            m.device() != t.device() || !m.is_contiguous())
            bad("credit: matrices must be contiguous tensors shaped like the input, of its dtype "
                "and on its device");
        return m.data_ptr();
    }
    // one fp32 value per row
    float* per_row(const at::Tensor& v) const {
        if (!v.defined()) bad("credit: the forward pass's mean and rstd are required");
        if (v.scalar_type() != at::kFloat || v.numel() != rows || v.device() != t.device() ||
            !v.is_contiguous())
            bad("credit: mean and rstd must be contiguous fp32 tensors on the input's device, one "
                "element per row");
        return static_cast<float*>(v.data_ptr());
    }
    at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
        return at::detail::empty_cuda(sizes, type, t.device(), c10::nullopt);
    }
    at::Tensor like() const { return empty(t.sizes(), t.scalar_type()); }
};

// gamma and beta of a call, and their one dtype.
credit_dtype_t params(const Input& x, const at::Tensor& gamma, const at::Tensor& beta) {
    credit_dtype_t code = CREDIT_F32;
    bool any = false;
    for (const at::Tensor* p : {&gamma, &beta}) {
        if (!p->defined()) continue;
        if (p->numel() != x.cols || p->device() != x.t.device() || !p->is_contiguous())
            bad("credit: parameters must be contiguous tensors of cols elements on the input's "
                "device");
        const credit_dtype_t c = code_of(*p);
        if (any && c != code) bad("credit: parameters must have one dtype");
        code = c;
        any = true;
    }
    return code;
}

// The caller's workspace, or one of the size the call needs.
at::Tensor workspace(const Input& x, credit_op_t op, int backward, const at::Tensor& given,
                     size_t* bytes, credit_status_t* status) {
    size_t need = 0;
    *status = g_workspace(op, backward, x.rows, x.cols, x.code, x.t.get_device(), &need);
    if (given.defined()) {
        if (given.device() != x.t.device() || !given.is_contiguous())
            bad("credit: workspace must be a contiguous tensor on the input's device");
        *bytes = given.nbytes();
        return given;
    }
    *bytes = need;
    if (*status != CREDIT_OK || need == 0) return at::Tensor();
    return x.empty({(int64_t)need}, at::kByte);
}

const credit_dropout_t* drop_of(PyObject* address) {
    return address == Py_None ? nullptr
                              : static_cast<const credit_dropout_t*>(PyLong_AsVoidPtr(address));
}

void* stream(const Input& x) { return c10::cuda::getCurrentCUDAStream(x.t.get_device()).stream(); }

PyObject* wrapped(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

// What every entry returns: the outputs as a tuple, or the status as an int.
template <typename... T> PyObject* result(credit_status_t st, const T&... outs) {
    if (st != CREDIT_OK) return PyLong_FromLong((long)st);
    PyObject* tuple = PyTuple_New(sizeof...(outs));
    if (!tuple) return nullptr;
    Py_ssize_t i = 0;
    bool ok = true;
    auto put = [&](const at::Tensor& t) {
        PyObject* o = ok ? wrapped(t) : nullptr;
        ok = ok && o;
        if (o) PyTuple_SET_ITEM(tuple, i, o);
        ++i;
    };
    (put(outs), ...);
    if (!ok) {
        Py_DECREF(tuple);
        return nullptr;
    }
    return tuple;
}

template <typename F> PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    HANDLE_TH_ERRORS
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "credit: wrong number of arguments");
        return nullptr;
    }
    if (!g_dropout) {
        PyErr_SetString(PyExc_RuntimeError, "credit: the library is not bound");
        return nullptr;
    }
    try {
        PyObject* r = f();
        return PyErr_Occurred() ? (Py_XDECREF(r), nullptr) : r;
    } catch (const Refused& e) {
        PyErr_SetString(e.type, e.message);
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// dropout(x, drop address, residual, out)
PyObject* py_dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        no_graph(a, {0, 2, 3});
        const Input x(a[0]);
        const at::Tensor &residual = tensor(a[2]), &given = tensor(a[3]);
        const void* rp = x.matrix(residual);
        void* given_p = x.matrix(given);
        const c10::cuda::CUDAGuard guard(x.t.device());
        const at::Tensor out = given.defined() ? given : x.like();
        const credit_status_t st = g_dropout(ptr(x.t), rp, given_p ? given_p : ptr(out), x.rows,
                                             x.cols, x.code, drop_of(a[1]), stream(x));
        if (st == CREDIT_OK) written({&given});
        return result(st, out);
    });
}

// norm_forward(op, x, gamma, beta, eps, residual, drop address, out, h out, workspace)
PyObject* py_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        no_graph(a, {1, 2, 3, 5, 7, 8});
        const credit_op_t op = (credit_op_t)PyLong_AsLong(a[0]);
        const Input x(a[1]);
        const at::Tensor &gamma = tensor(a[2]), &beta = tensor(a[3]), &residual = tensor(a[5]);
        const at::Tensor &out = tensor(a[7]), &h_out = tensor(a[8]);
        const credit_dtype_t pcode = params(x, gamma, beta);
        const double eps = PyFloat_AsDouble(a[4]);
        if (PyErr_Occurred()) return nullptr;
        const credit_dropout_t* drop = drop_of(a[6]);
        const void* rp = x.matrix(residual);
        x.matrix(out);
        x.matrix(h_out);
        const c10::cuda::CUDAGuard guard(x.t.device());
        size_t wb = 0;
        credit_status_t st;
        const at::Tensor ws = workspace(x, op, 0, tensor(a[9]), &wb, &st);
        if (st != CREDIT_OK) return result(st);
        const at::Tensor y = out.defined() ? out : x.like();
        // without residual and dropout h is x itself, and is not written, unless y
        // takes x's place
        const bool same = !residual.defined() && (!drop || drop->p == 0.0) && ptr(y) != ptr(x.t);
        const at::Tensor h = h_out.defined() ? h_out : same ? x.t : x.like();
        const at::IntArrayRef per_row = x.t.sizes().slice(0, x.t.dim() - 1);
        const at::Tensor rstd = x.empty(per_row, at::kFloat);
        const at::Tensor mean = op == CREDIT_LAYERNORM ? x.empty(per_row, at::kFloat) : at::Tensor();
        st = g_forward(op, ptr(x.t), rp, drop, ptr(y), h_out.defined() || !same ? ptr(h) : nullptr,
                       static_cast<float*>(ptr(mean)), static_cast<float*>(ptr(rstd)), x.rows, x.cols,
                       x.code, ptr(gamma), ptr(beta), pcode, (float)eps, ptr(ws), wb, stream(x));
        if (st == CREDIT_OK) written({&out, &h_out});
        return result(st, y, h, mean, rstd);
    });
}

// norm_backward(op, dy, h, mean, rstd, gamma, dh, drop address, need dresidual, dx, dresidual,
//               workspace, beta)
PyObject* py_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        no_graph(a, {1, 2, 3, 4, 5, 6, 9, 10, 12});
        const credit_op_t op = (credit_op_t)PyLong_AsLong(a[0]);
        const Input dy(a[1]);
        const at::Tensor &h = tensor(a[2]), &gamma = tensor(a[5]), &dh = tensor(a[6]);
        const at::Tensor &dx_given = tensor(a[9]), &dr_given = tensor(a[10]), &beta = tensor(a[12]);
        if (!h.defined()) bad("credit: h is required");
        const void *hp = dy.matrix(h), *dhp = dy.matrix(dh);
        const float* mp = op == CREDIT_LAYERNORM ? dy.per_row(tensor(a[3])) : nullptr;
        const float* sp = dy.per_row(tensor(a[4]));
        const credit_dtype_t pcode = params(dy, gamma, beta);
        const credit_dropout_t* drop = drop_of(a[7]);
        const int want = PyObject_IsTrue(a[8]);
        if (want < 0 || PyErr_Occurred()) return nullptr;
        dy.matrix(dx_given);
        dy.matrix(dr_given);
        const c10::cuda::CUDAGuard guard(dy.t.device());
        size_t wb = 0;
        credit_status_t st;
        const at::Tensor ws = workspace(dy, op, 1, tensor(a[11]), &wb, &st);
        if (st != CREDIT_OK) return result(st);
        const at::Tensor dx = dx_given.defined() ? dx_given : dy.like();
        at::Tensor dr = dr_given;
        if (!dr.defined() && want && drop && drop->p > 0.0) dr = dy.like();
        at::Tensor dgamma, dbeta;
        if (gamma.defined()) dgamma = dy.empty(gamma.sizes(), gamma.scalar_type());
        // beta's gradient is shaped like beta, or like gamma where only that is given
        const at::Tensor& like_beta = beta.defined() ? beta : gamma;
        if (op == CREDIT_LAYERNORM && like_beta.defined())
            dbeta = dy.empty(like_beta.sizes(), like_beta.scalar_type());
        st = g_backward(op, ptr(dy.t), dhp, hp, mp, sp, ptr(gamma), pcode, drop, ptr(dx), ptr(dr),
                        ptr(dgamma), ptr(dbeta), dy.rows, dy.cols, dy.code, ptr(ws), wb, stream(dy));
        if (st == CREDIT_OK) written({&dx_given, &dr_given});
        // without dropout the two gradients are one
        return result(st, dx, dr.defined() || !want ? dr : dx, dgamma, dbeta);
    });
}

// bind(addresses of credit_dropout, credit_norm_workspace, credit_norm_forward,
//      credit_norm_backward)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
        return nullptr;
    }
    g_dropout = reinterpret_cast<decltype(g_dropout)>(PyLong_AsVoidPtr(a[0]));
    g_workspace = reinterpret_cast<decltype(g_workspace)>(PyLong_AsVoidPtr(a[1]));
    g_forward = reinterpret_cast<decltype(g_forward)>(PyLong_AsVoidPtr(a[2]));
    g_backward = reinterpret_cast<decltype(g_backward)>(PyLong_AsVoidPtr(a[3]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

#define CREDIT_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {{"bind", CREDIT_FAST(py_bind), nullptr},
                           {"dropout", CREDIT_FAST(py_dropout), nullptr},
                           {"norm_forward", CREDIT_FAST(py_forward), nullptr},
                           {"norm_backward", CREDIT_FAST(py_backward), nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "credit_train_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_credit_train_torch(void) { return PyModule_Create(&g_module); }
