// torch_ops.cpp -- the calls of ops.py on torch tensors as a Python extension module: argument checks, allocation of the
// results and one call of the C library each.  At decode sizes a kernel runs for a few microseconds, and the
// same steps written in Python took 12 to 18 us a call against 4 to 5 here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace {

PyObject* g_error = nullptr;  // binding.MoeError

// Any refusal below: a Python error is set already.
struct Refused {};

[[noreturn]] void refuse(PyObject* kind, const char* what, const char* why) {
    PyErr_Format(kind, "%s: %s", what, why);
    throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, what, "a tensor expected");
    return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != nullptr && o != Py_None; }

moe_dtype dtype_of(const at::Tensor& t, const char* what) {
    switch (t.scalar_type()) {
        case at::kFloat: return MOE_F32;
        case at::kBFloat16: return MOE_BF16;
        case at::kHalf: return MOE_F16;
        default: refuse(PyExc_TypeError, what, "fp32, bf16 or fp16 expected");
    }
}

// Kernels run on the current device and its current stream: a tensor of another device is refused.
void here(const at::Tensor& t, const char* what) {
    c10::DeviceIndex current = -1;
    if (c10::cuda::GetDevice(&current) != cudaSuccess) current = -1;
    if (!t.is_cuda() || t.get_device() != current) refuse(PyExc_ValueError, what, "on another device than the current one");
}

// Row stride of a 2-D CUDA tensor whose rows are contiguous and do not overlap.
int64_t matrix(const at::Tensor& t, const char* what) {
    if (t.dim() != 2 || !t.is_cuda()) refuse(PyExc_ValueError, what, "a CUDA matrix expected");
    here(t, what);
    if (t.size(1) > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, what, "contiguous rows expected");
    if (t.size(0) <= 1) return t.size(1);
    if (t.stride(0) < t.size(1)) refuse(PyExc_ValueError, what, "rows may not overlap");
    return t.stride(0);
}

// A contiguous tensor of this type and shape (b < 0: one dimension) on `like`'s device.
const at::Tensor& plain(PyObject* o, at::ScalarType type, int64_t a, int64_t b, const at::Tensor& like, const char* what) {
    const at::Tensor& t = tensor(o, what);
    const bool shape = b < 0 ? t.dim() == 1 && t.size(0) == a : t.dim() == 2 && t.size(0) == a && t.size(1) == b;
    if (!shape || t.scalar_type() != type || t.device() != like.device() || !t.is_contiguous())
        refuse(PyExc_ValueError, what, "a contiguous tensor of the expected shape, type and device expected");
    return t;
}
template <typename T>
T* data(PyObject* o, at::ScalarType type, int64_t a, int64_t b, const at::Tensor& like, const char* what) {
    return given(o) ? static_cast<T*>(plain(o, type, a, b, like, what).data_ptr()) : nullptr;
}

// The bytes of a ctypes structure.
template <typename S>
const S* structure(PyObject* o, const char* what) {
    Py_buffer view;
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) throw Refused();
    const void* p = view.buf;
    const bool fits = view.len == (Py_ssize_t)sizeof(S);
    PyBuffer_Release(&view);  // (the caller's object lives through the call)
    if (!fits) refuse(PyExc_TypeError, what, "another structure expected");
    return static_cast<const S*>(p);
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v == 1;
}
int32_t narrow(int64_t v, const char* what) {
    if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, what, "too large");
    return (int32_t)v;
}

moe_stream_t stream() { return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }

at::Tensor fresh(int64_t a, int64_t b, at::ScalarType type, const at::Tensor& like) {
    const int64_t shape[2] = {a, b};
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

void check(moe_status s, const char* fn) {
    if (s == MOE_OK) return;
    PyObject* e = PyObject_CallFunction(g_error ? g_error : PyExc_RuntimeError, "si", fn, (int)s);
    if (e) {
        PyErr_SetObject((PyObject*)Py_TYPE(e), e);
        Py_DECREF(e);
    }
    throw Refused();
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* t = PyTuple_New(2);
    if (!t || !a || !b) {
        Py_XDECREF(t);
        Py_XDECREF(a);
        Py_XDECREF(b);
        throw Refused();
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    return t;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// route_scores(logits, k, rule, bias, scores, counts) -> ids, w
PyObject* route_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const at::Tensor& l = tensor(a[0], "logits");
        const int64_t ld = matrix(l, "logits"), T = l.size(0), E = l.size(1), k = integer(a[1]);
        const moe_dtype dt = dtype_of(l, "logits");
        const moe_route_rule* rule = structure<moe_route_rule>(a[2], "rule");
        const float* bias = data<float>(a[3], at::kFloat, E, -1, l, "bias");
        float* scores = data<float>(a[4], at::kFloat, T, E, l, "scores");
        int32_t* counts = data<int32_t>(a[5], at::kInt, E, -1, l, "counts");
        if (k < 0) refuse(PyExc_ValueError, "k", "negative");
        at::Tensor ids = fresh(T, k, at::kInt, l), w = fresh(T, k, at::kFloat, l);
        check(moe_route_scores(l.data_ptr(), dt, ld, bias, narrow(T, "T"), narrow(E, "E"), narrow(k, "k"), rule,
                               static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(w.data_ptr()), scores, counts, stream()),
              "moe_route_scores");
        return pair(wrap(ids), wrap(w));
    });
}

// route_scores_backward(logits, ids, dw, rule, dscores) -> dlogits
PyObject* route_scores_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        const at::Tensor& l = tensor(a[0], "logits");
        const int64_t ld = matrix(l, "logits"), T = l.size(0), E = l.size(1);
        const moe_dtype dt = dtype_of(l, "logits");
        const at::Tensor& ids0 = tensor(a[1], "ids");
        if (ids0.dim() != 2) refuse(PyExc_ValueError, "ids", "[T, k] expected");
        const int64_t k = ids0.size(1);
        const int32_t* ids = static_cast<const int32_t*>(plain(a[1], at::kInt, T, k, l, "ids").data_ptr());
        const float* dw = static_cast<const float*>(plain(a[2], at::kFloat, T, k, l, "dw").data_ptr());
        const moe_route_rule* rule = structure<moe_route_rule>(a[3], "rule");
        const float* dscores = data<float>(a[4], at::kFloat, T, E, l, "dscores");
        at::Tensor dl = fresh(T, E, l.scalar_type(), l);
        check(moe_route_scores_backward(l.data_ptr(), dt, ld, narrow(T, "T"), narrow(E, "E"), narrow(k, "k"), rule, ids, dw, dscores,
                                        dl.data_ptr(), E, stream()),
              "moe_route_scores_backward");
        return wrap(dl);
    });
}

// combine_backward(dy, y_perm, inv_pos, w, need_dw, need_dy_perm) -> dw, dy_perm
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const at::Tensor& dy = tensor(a[0], "dy");
        if (dy.dim() != 2 || !dy.is_cuda() || dy.scalar_type() != at::kBFloat16 || !dy.is_contiguous())
            refuse(PyExc_ValueError, "dy", "contiguous bf16 [T, d] on CUDA expected");
        here(dy, "dy");
        const at::Tensor& w0 = tensor(a[3], "w");
        if (w0.dim() != 2) refuse(PyExc_ValueError, "w", "[T, k] expected");
        const int64_t T = dy.size(0), d = dy.size(1), k = w0.size(1);
        const bool need_dw = truth(a[4]), need_dyp = truth(a[5]);
        const float* w = static_cast<const float*>(plain(a[3], at::kFloat, T, k, dy, "w").data_ptr());
        const int32_t* inv = static_cast<const int32_t*>(plain(a[2], at::kInt, T * k, -1, dy, "inv_pos").data_ptr());
        const uint16_t* yp = nullptr;
        if (need_dw) yp = static_cast<const uint16_t*>(plain(a[1], at::kBFloat16, T * k, d, dy, "y_perm").data_ptr());
        at::Tensor dw, dyp;
        if (need_dw) dw = fresh(T, k, at::kFloat, dy);
        if (need_dyp) dyp = fresh(T * k, d, at::kBFloat16, dy);
        if (need_dw || need_dyp)
            check(moe_combine_backward(static_cast<const uint16_t*>(dy.data_ptr()), yp, inv, w, narrow(T, "T"), narrow(k, "k"),
                                       narrow(d, "d"), need_dw ? static_cast<float*>(dw.data_ptr()) : nullptr,
                                       need_dyp ? static_cast<uint16_t*>(dyp.data_ptr()) : nullptr, stream()),
                  "moe_combine_backward");
        PyObject* first = need_dw ? wrap(dw) : (Py_INCREF(Py_None), Py_None);
        return pair(first, need_dyp ? wrap(dyp) : (Py_INCREF(Py_None), Py_None));
    });
}

// An operand as ops.py passes it: its structure, rows, K and device index.
struct Operand {
    const moe_nvfp4_operand* op = nullptr;
    int64_t rows = 0, K = 0;
};
Operand operand(PyObject* const* a, const at::Tensor& like, const char* what) {
    Operand o;
    if (!given(a[0])) return o;
    o.op = structure<moe_nvfp4_operand>(a[0], what);
    o.rows = integer(a[1]);
    o.K = integer(a[2]);
    if (integer(a[3]) != like.get_device()) refuse(PyExc_ValueError, what, "on another device than the tensors");
    return o;
}
void expect(const Operand& o, int64_t rows, int64_t K, const char* what) {
    if (o.rows == rows && o.K == K) return;
    PyErr_Format(PyExc_ValueError, "%s: an operand [%lld, %lld] expected, got [%lld, %lld]", what, (long long)rows, (long long)K,
                 (long long)o.rows, (long long)o.K);
    throw Refused();
}
struct Space {
    void* p = nullptr;
    size_t bytes = 0;
};
Space space(PyObject* o, const at::Tensor& like) {
    Space s;
    if (!given(o)) return s;
    const at::Tensor& t = tensor(o, "workspace");
    if (!t.is_contiguous() || t.device() != like.device()) refuse(PyExc_ValueError, "workspace", "a contiguous tensor on the same device expected");
    s.p = t.data_ptr();
    s.bytes = t.nbytes();
    return s;
}
// The result: `o`, or a new matrix of `type`.
at::Tensor output(PyObject* o, int64_t M, int64_t N, at::ScalarType type, const at::Tensor& like) {
    if (!given(o)) return fresh(M, N, type, like);
    const at::Tensor& t = tensor(o, "out");
    if (t.dim() != 2 || t.size(0) != M || t.size(1) != N || t.device() != like.device())
        refuse(PyExc_ValueError, "out", "[M, N] on the same device expected");
    return t;
}

// nvfp4_quantize(x, rows (4), cols (4), workspace, scales_given)
PyObject* nvfp4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const at::Tensor& x = tensor(a[0], "x");
        const int64_t ld = matrix(x, "x"), R = x.size(0), C = x.size(1);
        const moe_dtype dt = dtype_of(x, "x");
        const Operand rows = operand(a + 1, x, "rows"), cols = operand(a + 5, x, "cols");
        if (!rows.op && !cols.op) refuse(PyExc_ValueError, "rows or cols", "an operand to fill expected");
        if (rows.op) expect(rows, R, C, "rows");
        if (cols.op) expect(cols, C, R, "cols");
        const Space ws = space(a[9], x);
        check(moe_nvfp4_quantize(x.data_ptr(), dt, R, C, ld, rows.op, cols.op, truth(a[10]), ws.p, ws.bytes, stream()),
              "moe_nvfp4_quantize");
        Py_RETURN_NONE;
    });
}

// nvfp4_room(rows, K, device index) -> q, s, gs, their addresses: room for an operand with a scale per row
PyObject* nvfp4_room(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        const int64_t rows = integer(a[0]), K = integer(a[1]);
        const int64_t nq = (int64_t)moe_nvfp4_operand_codes(rows, K), ns = (int64_t)moe_nvfp4_operand_scales(rows, K);
        if (K < 1 || (nq == 0 && rows != 0)) refuse(PyExc_ValueError, "operand", "unsupported shape");
        const at::Device on(at::kCUDA, (c10::DeviceIndex)narrow(integer(a[2]), "device"));
        const at::Tensor q = at::detail::empty_cuda({nq}, at::kByte, on, std::nullopt), s = at::detail::empty_cuda({ns}, at::kByte, on, std::nullopt);
        const at::Tensor gs = at::detail::empty_cuda({rows}, at::kFloat, on, std::nullopt);
        return Py_BuildValue("NNNKKK", wrap(q), wrap(s), wrap(gs), (unsigned long long)reinterpret_cast<uintptr_t>(q.data_ptr()),
                             (unsigned long long)reinterpret_cast<uintptr_t>(s.data_ptr()),
                             (unsigned long long)reinterpret_cast<uintptr_t>(gs.data_ptr()));
    });
}

// nvfp4_matmul(a (4), b (4), like, workspace, out): like: a tensor whose type the result has, on the operands' device
PyObject* nvfp4_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const at::Tensor& like = tensor(a[8], "operand");
        here(like, "a, b");
        const Operand A = operand(a, like, "a"), B = operand(a + 4, like, "b");
        if (!A.op || !B.op) refuse(PyExc_ValueError, "a, b", "operands expected");
        expect(B, B.rows, A.K, "b");
        const at::ScalarType type = static_cast<at::ScalarType>(integer(a[9]));
        const Space ws = space(a[10], like);
        at::Tensor y = output(a[11], A.rows, B.rows, type, like);
        if (y.scalar_type() != type) refuse(PyExc_ValueError, "out", "another type expected");
        check(moe_nvfp4_matmul(A.op, B.op, A.rows, B.rows, A.K, y.data_ptr(), dtype_of(y, "out"), matrix(y, "out"), ws.p, ws.bytes, stream()),
              "moe_nvfp4_matmul");
        return wrap(y);
    });
}

// nvfp4_linear(x, W (4), workspace, out) -> y
PyObject* nvfp4_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor& x = tensor(a[0], "x");
        const int64_t ld = matrix(x, "x"), M = x.size(0), K = x.size(1);
        const moe_dtype dt = dtype_of(x, "x");
        const Operand W = operand(a + 1, x, "W");
        if (!W.op) refuse(PyExc_ValueError, "W", "an operand expected");
        expect(W, W.rows, K, "W");
        const Space ws = space(a[5], x);
        at::Tensor y = output(a[6], M, W.rows, x.scalar_type(), x);
        check(moe_nvfp4_linear(x.data_ptr(), dt, M, K, ld, W.op, W.rows, y.data_ptr(), dtype_of(y, "out"), matrix(y, "out"), ws.p,
                               ws.bytes, stream()),
              "moe_nvfp4_linear");
        return wrap(y);
    });
}

PyObject* set_error(PyObject*, PyObject* kind) {
    Py_XDECREF(g_error);
    Py_INCREF(kind);
    g_error = kind;
    Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(route_scores), FAST(route_scores_backward), FAST(combine_backward), FAST(nvfp4_quantize), FAST(nvfp4_room),
                         FAST(nvfp4_matmul), FAST(nvfp4_linear), {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "moe_torch_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_moe_torch_ops(void) { return PyModule_Create(&module); }
