// Python binding of the decode-side operators and of those that train and
// quantise (include/omm.h): argument
// marshalling only, as _omm.py does it for the others, but without ctypes.
// These operators run for a few microseconds, and describing seven tensors and
// allocating the outputs from Python takes longer than that (moe_route of one
// token: 9.8 us a call through ctypes with packed descriptors, 2.3 us of kernel).
//
// Every function returns its outputs or raises: TypeError / ValueError for
// tensors that cannot be described, OmmError for a status of the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include "omm.h"

namespace {

struct Lib {
    decltype(&omm_lora_matmul) lora_matmul;
    decltype(&omm_lora_matmul_workspace_size) lora_matmul_ws;
    decltype(&omm_moe_route) moe_route;
    decltype(&omm_moe_layer) moe_layer;
    decltype(&omm_moe_layer_workspace_size) moe_layer_ws;
    decltype(&omm_token_logprobs) token_logprobs;
    decltype(&omm_token_logprobs_workspace_size) token_logprobs_ws;
    decltype(&omm_token_logprobs_grad) token_logprobs_grad;
    decltype(&omm_quantize_rows) quantize_rows;
    decltype(&omm_int8_matmul) int8_matmul;
    decltype(&omm_int8_matmul_workspace_size) int8_matmul_ws;
    decltype(&omm_moe_balance) moe_balance;
    decltype(&omm_moe_balance_workspace_size) moe_balance_ws;
    decltype(&omm_moe_route_grad) moe_route_grad;
    decltype(&omm_orthogonalize) orthogonalize;
    decltype(&omm_orthogonalize_workspace_size) orthogonalize_ws;
} L = {};
PyObject* omm_error = nullptr;

int dtype_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return OMM_F32;
        case at::kHalf: return OMM_F16;
        case at::kBFloat16: return OMM_BF16;
        case at::kDouble: return OMM_F64;
        case at::kChar: return OMM_I8;
        case at::kByte: return OMM_U8;
        case at::kInt: return OMM_I32;
        case at::kLong: return OMM_I64;
        default: return -1;
    }
}

struct Failed {};  // a Python error is set

[[noreturn]] void fail(PyObject* type, const char* what) {
    PyErr_SetString(type, what);
    throw Failed{};
}

const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "expected a torch.Tensor");
    return THPVariable_Unpack(o);
}

omm_tensor describe(const at::Tensor& x) {
    if (!x.is_cuda()) fail(PyExc_ValueError, "tensor must be on the GPU");
    if (!x.is_contiguous()) fail(PyExc_ValueError, "tensor must be contiguous (row-major)");
    if (x.dim() > OMM_MAX_DIMS) fail(PyExc_ValueError, "too many dims");
    omm_tensor t = {};
    t.dtype = dtype_of(x.scalar_type());
    if (t.dtype < 0) fail(PyExc_TypeError, "tensor of an unsupported dtype");
    t.data = x.numel() > 0 ? x.data_ptr() : nullptr;
    t.ndim = (int32_t)x.dim();
    for (int64_t i = 0; i < x.dim(); ++i) t.shape[i] = x.size(i);
    return t;
}

// a tensor argument (None: no tensor) with its descriptor
struct Arg {
    omm_tensor t;
    const omm_tensor* p = nullptr;
    explicit Arg(PyObject* o) {
        if (o == Py_None) return;
        t = describe(tensor(o));
        p = &t;
    }
    Arg(const Arg&) = delete;
};

struct Out {
    at::Tensor x;
    omm_tensor t;
    // the caller's tensor, or a new one of this shape
    Out(PyObject* o, at::IntArrayRef shape, const at::Tensor& like, at::ScalarType dt)
        : x(o && o != Py_None ? tensor(o) : at::empty(shape, like.options().dtype(dt))), t(describe(x)) {}
};

struct Workspace {
    at::Tensor x;
    Workspace(PyObject* o, const at::Tensor& like, size_t (*need)(const void*), const void* arg)
        : x(o != Py_None ? tensor(o)
                         : at::empty({(int64_t)std::max<size_t>(need(arg), 256)}, like.options().dtype(at::kByte))) {
        if (!x.is_cuda() || !x.is_contiguous()) fail(PyExc_ValueError, "workspace must be a contiguous GPU tensor");
    }
    void* ptr() const { return x.data_ptr(); }
    size_t bytes() const { return x.nbytes(); }
};
template <typename F>
Workspace workspace(PyObject* o, const at::Tensor& like, const F& need) {
    return Workspace(o, like, [](const void* f) { return (*(const F*)f)(); }, &need);
}

int integer(PyObject* o) {  // OverflowError for what the library's int does not hold
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    if (v != (int)v) fail(PyExc_OverflowError, "integer argument out of range");
    return (int)v;
}

// The current stream of x's device, to which what is allocated here belongs too.
// (A call for another stream makes that one current: memory of this stream's could
// be handed out again while the other one still uses it.)
void* stream(const at::Tensor& x) { return (void*)c10::hip::getCurrentHIPStream(x.device().index()).stream(); }

template <typename F>
void call(const char* what, F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f();
    Py_END_ALLOW_THREADS;
    if (!rc) return;
    PyObject* e = PyObject_CallFunction(omm_error, "is", rc, what);
    if (e) {
        PyErr_SetObject(omm_error, e);
        Py_DECREF(e);
    }
    throw Failed{};
}

// no C++ exception leaves through the C entry
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    if (!omm_error) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
        return nullptr;
    }
    try {
        return f();
    } catch (const Failed&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject* pack(std::initializer_list<at::Tensor> xs) {
    PyObject* t = PyTuple_New((Py_ssize_t)xs.size());
    if (!t) throw Failed{};
    Py_ssize_t i = 0;
    for (const at::Tensor& x : xs) PyTuple_SET_ITEM(t, i++, THPVariable_Wrap(x));
    return t;
}

// X, W, A, B, adapter_indices, adapter_scale, bias, trans, Y, workspace
PyObject* lora_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &X = tensor(a[0]), &W = tensor(a[1]), &A = tensor(a[2]);
        const int trans = integer(a[7]);
        if (X.dim() != 2 || W.dim() != 2 || A.dim() != 3) fail(PyExc_ValueError, "X and W must be 2-d, A 3-d");
        Arg x(a[0]), w(a[1]), la(a[2]), lb(a[3]), idx(a[4]), scale(a[5]), bias(a[6]);
        const int64_t M = X.size(0), K = X.size(1), N = W.size(trans ? 0 : 1), R = A.size(trans ? 1 : 2);
        Out y(a[8], {M, N}, X, X.scalar_type());
        const Workspace ws = workspace(a[9], X, [&] { return L.lora_matmul_ws(M, K, N, R, x.t.dtype); });
        void* s = stream(X);
        call("omm_lora_matmul", [&] {
            return L.lora_matmul(x.p, w.p, la.p, lb.p, idx.p, scale.p, bias.p, trans, &y.t, ws.ptr(), ws.bytes(), s);
        });
        return pack({y.x, ws.x});
    });
}

// logits, top_k, renormalize, indices, weights
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const at::Tensor& logits = tensor(a[0]);
        const int k = integer(a[1]), renorm = integer(a[2]);
        if (logits.dim() != 2) fail(PyExc_ValueError, "logits must be 2-d");
        Arg x(a[0]);
        const int64_t M = logits.size(0), kk = std::max(k, 0);
        Out ids(a[3], {M, kk}, logits, at::kInt), w(a[4], {M, kk}, logits, at::kFloat);
        void* s = stream(logits);
        call("omm_moe_route", [&] { return L.moe_route(x.p, k, renorm, &ids.t, &w.t, s); });
        return pack({ids.x, w.x});
    });
}

// X, router_logits, top_k, W_gate, W_up, W_down, renormalize, activation, trans, Y, workspace
PyObject* moe_layer(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const at::Tensor &X = tensor(a[0]), &W = tensor(a[3]);
        const int k = integer(a[2]), renorm = integer(a[6]), act = integer(a[7]), trans = integer(a[8]);
        if (X.dim() != 2 || W.dim() != 3) fail(PyExc_ValueError, "X must be 2-d, the weights 3-d");
        Arg x(a[0]), logits(a[1]), wg(a[3]), wu(a[4]), wd(a[5]);
        const int64_t M = X.size(0), K = X.size(1), E = W.size(0), F = W.size(trans ? 1 : 2);
        Out y(a[9], {M, K}, X, X.scalar_type());
        const Workspace ws = workspace(a[10], X, [&] { return L.moe_layer_ws(M, K, F, E, k); });
        void* s = stream(X);
        call("omm_moe_layer", [&] {
            return L.moe_layer(x.p, logits.p, k, renorm, wg.p, wu.p, wd.p, act, trans, &y.t, ws.ptr(), ws.bytes(), s);
        });
        return pack({y.x, ws.x});
    });
}

// logits, targets, top_k, workspace
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        const at::Tensor& logits = tensor(a[0]);
        const int k = integer(a[2]);
        const int64_t kk = std::max(k, 0);
        if (logits.dim() != 2) fail(PyExc_ValueError, "logits must be 2-d");
        Arg x(a[0]), t(a[1]);
        const int64_t M = logits.size(0), V = logits.size(1);
        Out lp(nullptr, {M}, logits, at::kFloat), ent(nullptr, {M}, logits, at::kFloat),
            lse(nullptr, {M}, logits, at::kFloat), ids(nullptr, {M, kk}, logits, at::kInt),
            tlp(nullptr, {M, kk}, logits, at::kFloat);
        const Workspace ws = workspace(a[3], logits, [&] { return L.token_logprobs_ws(M, V, k); });
        void* s = stream(logits);
        call("omm_token_logprobs", [&] {
            return L.token_logprobs(x.p, t.p, k, &lp.t, &ent.t, &lse.t, &ids.t, &tlp.t, ws.ptr(), ws.bytes(), s);
        });
        return pack({lp.x, ent.x, lse.x, ids.x, tlp.x});
    });
}

// logits, targets, lse, entropy, grad_logprobs, grad_entropy, grad_logits
PyObject* token_logprobs_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor& logits = tensor(a[0]);
        Arg x(a[0]), t(a[1]), lse(a[2]), ent(a[3]), gl(a[4]), gh(a[5]);
        Out g(a[6], logits.sizes(), logits, logits.scalar_type());
        void* s = stream(logits);
        call("omm_token_logprobs_grad",
             [&] { return L.token_logprobs_grad(x.p, t.p, lse.p, ent.p, gl.p, gh.p, &g.t, s); });
        return THPVariable_Wrap(g.x);
    });
}

// The device of the first tensor, current while the call's memory and kernels are
// made, and the only one that its other tensors may be on.
struct On {
    const at::Tensor& x;
    c10::DeviceGuard guard;
    On(PyObject* first, std::initializer_list<PyObject*> others) : x(gpu(first)), guard(x.device()) {
        for (PyObject* o : others)
            if (o != Py_None && tensor(o).device() != x.device()) fail(PyExc_ValueError, "tensors are on different devices");
    }
    static const at::Tensor& gpu(PyObject* o) {
        const at::Tensor& x = tensor(o);
        if (!x.is_cuda()) fail(PyExc_ValueError, "tensor must be on the GPU");
        return x;
    }
};

// a mask: bytes, or torch.bool, which is a byte of 0 or 1
struct Mask {
    omm_tensor t;
    const omm_tensor* p = nullptr;
    explicit Mask(PyObject* o) {
        if (o == Py_None) return;
        const at::Tensor& x = tensor(o);
        t = describe(x.scalar_type() == at::kBool ? x.view(at::kByte) : x);
        p = &t;
    }
    Mask(const Mask&) = delete;
};

// X, Q, scale
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&] {
        const On on(a[0], {a[1], a[2]});
        if (on.x.dim() != 2) fail(PyExc_ValueError, "X must be 2-d");
        Arg x(a[0]);
        Out q(a[1], on.x.sizes(), on.x, at::kChar), scale(a[2], {on.x.size(0)}, on.x, at::kFloat);
        void* s = stream(on.x);
        call("omm_quantize_rows", [&] { return L.quantize_rows(x.p, &q.t, &scale.t, s); });
        return pack({q.x, scale.x});
    });
}

// a, a_scale, b, b_scale, bias, dtype of Y, Y, workspace
PyObject* int8_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        const On on(a[0], {a[1], a[2], a[3], a[4], a[6], a[7]});
        const at::Tensor &X = on.x, &W = tensor(a[2]);
        if (X.dim() != 2 || W.dim() != 2) fail(PyExc_ValueError, "a and b must be 2-d");
        Arg x(a[0]), xs(a[1]), w(a[2]), ws_(a[3]), bias(a[4]);
        const int dt = integer(a[5]);
        if (dt != OMM_F32 && dt != OMM_F16 && dt != OMM_BF16) fail(PyExc_ValueError, "Y is bfloat16, float16 or float32");
        const at::ScalarType yt = dt == OMM_F32 ? at::kFloat : dt == OMM_F16 ? at::kHalf : at::kBFloat16;
        const int64_t M = X.size(0), K = X.size(1), N = W.size(0);
        Out y(a[6], {M, N}, X, yt);
        if (a[7] == Py_None && L.int8_matmul_ws(M, K, N, x.t.dtype) == 0) {
            void* s = stream(X);
            call("omm_int8_matmul", [&] { return L.int8_matmul(x.p, xs.p, w.p, ws_.p, bias.p, &y.t, nullptr, 0, s); });
            return pack({y.x, at::Tensor()});
        }
        const Workspace ws = workspace(a[7], X, [&] { return L.int8_matmul_ws(M, K, N, x.t.dtype); });
        void* s = stream(X);
        call("omm_int8_matmul",
             [&] { return L.int8_matmul(x.p, xs.p, w.p, ws_.p, bias.p, &y.t, ws.ptr(), ws.bytes(), s); });
        return pack({y.x, ws.x});
    });
}

// logits, indices, token_mask, workspace
PyObject* moe_balance(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        const On on(a[0], {a[1], a[2], a[3]});
        const at::Tensor& logits = on.x;
        if (logits.dim() != 2) fail(PyExc_ValueError, "logits must be 2-d");
        Arg x(a[0]), ids(a[1]);
        Mask mask(a[2]);
        const int64_t M = logits.size(0), E = logits.size(1);
        Out losses(nullptr, {2}, logits, at::kFloat), counts(nullptr, {E}, logits, at::kInt),
            tokens(nullptr, {1}, logits, at::kInt);
        void* s = stream(logits);
        const auto run = [&](void* ws, size_t bytes) {
            call("omm_moe_balance", [&] {
                return L.moe_balance(x.p, ids.p, mask.p, &losses.t, &counts.t, &tokens.t, ws, bytes, s);
            });
            return pack({losses.x, counts.x, tokens.x});
        };
        if (a[3] == Py_None && L.moe_balance_ws(M, E) == 0) return run(nullptr, 0);
        const Workspace ws = workspace(a[3], logits, [&] { return L.moe_balance_ws(M, E); });
        return run(ws.ptr(), ws.bytes());
    });
}

// logits, indices, grad_weights, renormalize, token_mask, counts, tokens, grad_losses, grad_logits
PyObject* moe_route_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const On on(a[0], {a[1], a[2], a[4], a[5], a[6], a[7], a[8]});
        Arg x(a[0]), ids(a[1]), gw(a[2]), counts(a[5]), tokens(a[6]), gl(a[7]);
        Mask mask(a[4]);
        const int renorm = integer(a[3]);
        Out g(a[8], on.x.sizes(), on.x, on.x.scalar_type());
        void* s = stream(on.x);
        call("omm_moe_route_grad",
             [&] { return L.moe_route_grad(x.p, ids.p, gw.p, renorm, mask.p, counts.p, tokens.p, gl.p, &g.t, s); });
        return THPVariable_Wrap(g.x);
    });
}

// G, steps, out, workspace
PyObject* orthogonalize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        const On on(a[0], {a[2], a[3]});
        const at::Tensor& G = on.x;
        const int steps = integer(a[1]);
        if (G.dim() != 2 && G.dim() != 3) fail(PyExc_ValueError, "G must be 2-d, or 3-d for a batch");
        Arg g(a[0]);
        Out out(a[2], G.sizes(), G, G.scalar_type());
        const int d = (int)G.dim() - 2;
        const Workspace ws =
            workspace(a[3], G, [&] { return L.orthogonalize_ws(d ? G.size(0) : 1, G.size(d), G.size(d + 1)); });
        void* s = stream(G);
        call("omm_orthogonalize", [&] { return L.orthogonalize(g.p, steps, &out.t, ws.ptr(), ws.bytes(), s); });
        return pack({out.x, ws.x});
    });
}

// load(path of libomm.so, OmmError)
PyObject* load(PyObject*, PyObject* args) {
    const char* path;
    PyObject* error;
    if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
    void* h = dlopen(path, RTLD_NOW);
    if (!h) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    const struct {
        void** f;
        const char* name;
    } table[] = {
        {(void**)&L.lora_matmul, "omm_lora_matmul"},
        {(void**)&L.lora_matmul_ws, "omm_lora_matmul_workspace_size"},
        {(void**)&L.moe_route, "omm_moe_route"},
        {(void**)&L.moe_layer, "omm_moe_layer"},
        {(void**)&L.moe_layer_ws, "omm_moe_layer_workspace_size"},
        {(void**)&L.token_logprobs, "omm_token_logprobs"},
        {(void**)&L.token_logprobs_ws, "omm_token_logprobs_workspace_size"},
        {(void**)&L.token_logprobs_grad, "omm_token_logprobs_grad"},
        {(void**)&L.quantize_rows, "omm_quantize_rows"},
        {(void**)&L.int8_matmul, "omm_int8_matmul"},
        {(void**)&L.int8_matmul_ws, "omm_int8_matmul_workspace_size"},
        {(void**)&L.moe_balance, "omm_moe_balance"},
        {(void**)&L.moe_balance_ws, "omm_moe_balance_workspace_size"},
        {(void**)&L.moe_route_grad, "omm_moe_route_grad"},
        {(void**)&L.orthogonalize, "omm_orthogonalize"},
        {(void**)&L.orthogonalize_ws, "omm_orthogonalize_workspace_size"},
    };
    for (const auto& e : table)
        if (!(*e.f = dlsym(h, e.name))) {
            PyErr_Format(PyExc_RuntimeError, "%s lacks %s", path, e.name);
            return nullptr;
        }
    Py_INCREF(error);
    Py_XDECREF(omm_error);
    omm_error = error;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"load", load, METH_VARARGS, nullptr},
    {"lora_matmul", (PyCFunction)(void (*)())lora_matmul, METH_FASTCALL, nullptr},
    {"moe_route", (PyCFunction)(void (*)())moe_route, METH_FASTCALL, nullptr},
    {"moe_layer", (PyCFunction)(void (*)())moe_layer, METH_FASTCALL, nullptr},
    {"token_logprobs", (PyCFunction)(void (*)())token_logprobs, METH_FASTCALL, nullptr},
    {"token_logprobs_grad", (PyCFunction)(void (*)())token_logprobs_grad, METH_FASTCALL, nullptr},
    {"quantize_rows", (PyCFunction)(void (*)())quantize_rows, METH_FASTCALL, nullptr},
    {"int8_matmul", (PyCFunction)(void (*)())int8_matmul, METH_FASTCALL, nullptr},
    {"moe_balance", (PyCFunction)(void (*)())moe_balance, METH_FASTCALL, nullptr},
    {"moe_route_grad", (PyCFunction)(void (*)())moe_route_grad, METH_FASTCALL, nullptr},
    {"orthogonalize", (PyCFunction)(void (*)())orthogonalize, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
