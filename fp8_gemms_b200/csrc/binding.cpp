// binding.cpp -- the calls of the operators between the GEMMs as a Python module: checks of
// the arguments, allocation of outputs and workspaces, and the C call (include/lm_fp8.h)
// on the current stream of the tensors' device.  Small calls are bound by the host: a
// layer norm of 16 x 1024 takes 2 us on the GPU and 6.0 us here, of which about 3 are the
// three allocations and 3 the launch; through Python and ctypes it was 14.7.
//
// What a call cannot run it refuses with the exception type that use_error() was given
// (LmError), made from the C interface's status and a text.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <string>

#include "lm_fp8.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;

[[noreturn]] void refuse(const char* what, const char* why, int status = LM_ERR_INVALID_ARG) {
    const std::string text = *why ? std::string(what) + ": " + why : std::string(what);
    if (PyObject* e = PyObject_CallFunction(g_error, "is", status, text.c_str())) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

// Runs without the interpreter's lock: an allocation can wait for the GPU, and a launch
// waits while the queue is full.
template <typename F>
auto unlocked(F f) {
    struct Lock {
        PyThreadState* state = PyEval_SaveThread();
        ~Lock() { PyEval_RestoreThread(state); }
    } lock;
    return f();
}

template <typename F>
void call(const char* what, F f) {
    const lm_status st = unlocked(f);
    if (st != LM_OK) refuse(what, "", st);
}

// A tensor argument; None gives an undefined one.
const Tensor& tensor(const char* what, PyObject* o) {
    static const Tensor none;
    if (o == Py_None) return none;
    if (!THPVariable_Check(o)) refuse(what, "a tensor is wanted");
    return THPVariable_Unpack(o);
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v;
}
// Any integer, as also `start` of rope() is taken (Python's, numpy's, a tensor's).
uint64_t unsigned64(const char* what, PyObject* o) {
    THPObjectPtr i(PyNumber_Index(o));
    const unsigned long long v = i ? PyLong_AsUnsignedLongLong(i.get()) : 0;
    if (PyErr_Occurred()) {
        if (!PyErr_ExceptionMatches(PyExc_TypeError) && !PyErr_ExceptionMatches(PyExc_OverflowError))
            throw python_error();
        PyErr_Clear();
        refuse(what, "offset is an unsigned 64-bit integer");
    }
    return v;
}

template <typename T = void>
T* ptr(const Tensor& t) {
    return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

// Uninitialised tensors, without the dispatcher on the way (0.4 us each).
Tensor new_like(const Tensor& x) {
    return unlocked([&]() -> Tensor {
        if (!x.is_non_overlapping_and_dense()) return at::empty_like(x);
        return Tensor(at::detail::empty_strided_cuda(x.sizes(), x.strides(), x.scalar_type(),
                                                     x.device()));
    });
}
Tensor new_vector(int64_t n, at::ScalarType type, at::Device device) {
    return unlocked([&] {
        return Tensor(at::detail::empty_cuda({n}, type, device, std::nullopt));
    });
}

// The first tensor of a call; the others share its sizes, type and device.
struct Rows {
    const char* what;
    Tensor x;
    int64_t rows, cols, ld;
    lm_dtype dtype;
    c10::cuda::OptionalCUDAGuard guard;

    Rows(const char* what_, const Tensor& t) : what(what_), x(t) {
        if (!x.defined() || x.dim() != 2 || !x.is_cuda()) refuse(what, "a 2-D CUDA tensor is wanted");
        dtype = x.scalar_type() == at::kBFloat16 ? LM_DTYPE_BF16 : LM_DTYPE_F32;
        if (dtype == LM_DTYPE_F32 && x.scalar_type() != at::kFloat)
            refuse(what, "bf16 or fp32 is wanted", LM_ERR_UNSUPPORTED_FORMAT);
        rows = x.size(0), cols = x.size(1);
        ld = stride_of(x);
        guard.set_device(x.device());
    }
    int64_t stride_of(const Tensor& t) const {
        if (cols > 1 && t.stride(1) != 1) refuse(what, "adjacent columns are wanted");
        return t.stride(0);
    }
    // The row stride of another tensor; 0 where it is left out.
    int64_t also(const Tensor& t) const {
        if (!t.defined()) return 0;
        if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols ||
            t.scalar_type() != x.scalar_type() || t.device() != x.device())
            refuse(what, "tensors of one shape, type and device are wanted");
        return stride_of(t);
    }
    void vector(const Tensor& t, int64_t n, at::ScalarType type) const {
        if (t.defined() && (t.dim() != 1 || t.size(0) != n || t.scalar_type() != type ||
                            t.device() != x.device() || !t.is_contiguous()))
            refuse(what, "a contiguous vector of another length, type or device is wanted");
    }
    const uint64_t* rng(const Tensor& t) const {
        if (!t.defined() || (t.scalar_type() != at::kLong && t.scalar_type() != at::kUInt64) ||
            t.numel() != 2 || t.device() != x.device() || !t.is_contiguous())
            refuse(what, "rng is a contiguous 64-bit integer {seed, offset} of the same device");
        return ptr<const uint64_t>(t);
    }
    Tensor like() const { return new_like(x); }
    Tensor fresh(int64_t n, at::ScalarType type) const { return new_vector(n, type, x.device()); }
    lm_stream_t stream() const {
        return c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
    }
};

template <typename... Ts>
PyObject* tuple(const Ts&... ts) {
    PyObject* out = PyTuple_New(sizeof...(ts));
    if (!out) throw python_error();
    int i = 0;
    (PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(ts)), ...);
    return out;
}

void count(const char* what, Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse(what, "another number of arguments is wanted");
}

// (x, weight, bias, eps, out, amax_out) -> (y, mean, rstd)
PyObject* layernorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char* what = "lm_layernorm_fwd";
    count(what, n, 6);
    Rows r(what, tensor(what, a[0]));
    const Tensor &w = tensor(what, a[1]), &b = tensor(what, a[2]), &amax = tensor(what, a[5]);
    r.vector(w, r.cols, r.x.scalar_type());
    r.vector(b, r.cols, r.x.scalar_type());
    r.vector(amax, 1, at::kFloat);
    Tensor y = tensor(what, a[4]);
    if (!y.defined()) y = r.like();
    const int64_t ldy = r.also(y);
    const Tensor mean = r.fresh(r.rows, at::kFloat), rstd = r.fresh(r.rows, at::kFloat);
    const float eps = (float)number(a[3]);
    call(what, [&] {
        return lm_layernorm_fwd(ptr(r.x), r.ld, ptr(w), ptr(b), r.rows, r.cols, eps, r.dtype,
                                ptr(y), ldy, ptr<float>(mean), ptr<float>(rstd), ptr<float>(amax),
                                r.stream());
    });
    return tuple(y, mean, rstd);
    END_HANDLE_TH_ERRORS
}

// dweight and dbias of a backward (made where they are left out and not accumulated), and
// its workspace.
struct Wgrads {
    Tensor w, b, ws;
    size_t bytes;
    uint32_t flags;
    Wgrads(const Rows& r, PyObject* dweight, PyObject* dbias, PyObject* accumulate)
        : w(tensor(r.what, dweight)), b(tensor(r.what, dbias)) {
        const bool sum = truth(accumulate);
        const at::ScalarType type = sum ? at::kFloat : r.x.scalar_type();
        flags = sum ? LM_NORM_ACCUMULATE_WGRAD : 0;
        r.vector(w, r.cols, type);
        r.vector(b, r.cols, type);
        if (!sum && !w.defined()) w = r.fresh(r.cols, type);
        if (!sum && !b.defined()) b = r.fresh(r.cols, type);
        bytes = lm_layernorm_workspace_size(r.rows, r.cols);
        ws = r.fresh((int64_t)bytes, at::kByte);
    }
};

// (dy, x, weight, mean, rstd, out, dweight, dbias, accumulate) -> (dx, dweight, dbias)
PyObject* layernorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char* what = "lm_layernorm_bwd";
    count(what, n, 9);
    Rows r(what, tensor(what, a[1]));
    const Tensor &dy = tensor(what, a[0]), &w = tensor(what, a[2]), &mean = tensor(what, a[3]),
                 &rstd = tensor(what, a[4]);
    const int64_t lddy = r.also(dy);
    r.vector(w, r.cols, r.x.scalar_type());
    r.vector(mean, r.rows, at::kFloat);
    r.vector(rstd, r.rows, at::kFloat);
    Tensor dx = tensor(what, a[5]);
    if (!dx.defined()) dx = r.like();
    const int64_t lddx = r.also(dx);
    const Wgrads g(r, a[6], a[7], a[8]);
    call(what, [&] {
        return lm_layernorm_bwd(ptr(dy), lddy, ptr(r.x), r.ld, ptr(w), ptr<float>(mean),
                                ptr<float>(rstd), r.rows, r.cols, r.dtype, ptr(dx), lddx,
                                ptr(g.w), ptr(g.b), ptr(g.ws), g.bytes, g.flags, r.stream());
    });
    return tuple(dx, g.w, g.b);
    END_HANDLE_TH_ERRORS
}

// (x, p, rng, offset, residual, out) -> y
PyObject* dropout_add(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char* what = "lm_dropout_add_fwd";
    count(what, n, 6);
    Rows r(what, tensor(what, a[0]));
    const Tensor& res = tensor(what, a[4]);
    const int64_t ldr = r.also(res);
    Tensor y = tensor(what, a[5]);
    if (!y.defined()) y = r.like();
    const int64_t ldy = r.also(y);
    const double p = number(a[1]);
    const uint64_t *rng = r.rng(tensor(what, a[2])), offset = unsigned64(what, a[3]);
    call(what, [&] {
        return lm_dropout_add_fwd(ptr(r.x), r.ld, ptr(res), ldr, r.rows, r.cols, r.dtype, p, rng,
                                  offset, ptr(y), ldy, r.stream());
    });
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// (dy, p, rng, offset, out) -> dx
PyObject* dropout_add_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char* what = "lm_dropout_add_bwd";
    count(what, n, 5);
    Rows r(what, tensor(what, a[0]));
    Tensor dx = tensor(what, a[4]);
    if (!dx.defined()) dx = r.like();
    const int64_t lddx = r.also(dx);
    const double p = number(a[1]);
    const uint64_t *rng = r.rng(tensor(what, a[2])), offset = unsigned64(what, a[3]);
    call(what, [&] {
        return lm_dropout_add_bwd(ptr(r.x), r.ld, r.rows, r.cols, r.dtype, p, rng, offset,
                                  ptr(dx), lddx, r.stream());
    });
    return THPVariable_Wrap(dx);
    END_HANDLE_TH_ERRORS
}

// (x, residual, weight, bias, p, rng, offset, eps, amax_out) -> (s, y, mean, rstd)
PyObject* dropout_add_layernorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char* what = "lm_dropout_add_layernorm_fwd";
    count(what, n, 9);
    Rows r(what, tensor(what, a[0]));
    const Tensor &res = tensor(what, a[1]), &w = tensor(what, a[2]), &b = tensor(what, a[3]),
                 &amax = tensor(what, a[8]);
    const int64_t ldr = r.also(res);
    r.vector(w, r.cols, r.x.scalar_type());
    r.vector(b, r.cols, r.x.scalar_type());
    r.vector(amax, 1, at::kFloat);
    const Tensor s = r.like(), y = r.like();
    const Tensor mean = r.fresh(r.rows, at::kFloat), rstd = r.fresh(r.rows, at::kFloat);
    const int64_t lds = r.also(s), ldy = r.also(y);
    const float eps = (float)number(a[7]);
    const double p = number(a[4]);
    const uint64_t *rng = r.rng(tensor(what, a[5])), offset = unsigned64(what, a[6]);
    call(what, [&] {
        return lm_dropout_add_layernorm_fwd(
            ptr(r.x), r.ld, ptr(res), ldr, ptr(w), ptr(b), r.rows, r.cols, eps, r.dtype, p, rng,
            offset, ptr(s), lds, ptr(y), ldy, ptr<float>(mean), ptr<float>(rstd), ptr<float>(amax),
            r.stream());
    });
    return tuple(s, y, mean, rstd);
    END_HANDLE_TH_ERRORS
}

// (dy, ds, s, weight, mean, rstd, p, rng, offset, dweight, dbias, accumulate)
// -> (dx, dresidual, dweight, dbias)
PyObject* dropout_add_layernorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char* what = "lm_dropout_add_layernorm_bwd";
    count(what, n, 12);
    Rows r(what, tensor(what, a[2]));
    const Tensor &dy = tensor(what, a[0]), &ds = tensor(what, a[1]), &w = tensor(what, a[3]),
                 &mean = tensor(what, a[4]), &rstd = tensor(what, a[5]);
    const int64_t lddy = r.also(dy), ldds = r.also(ds);
    r.vector(w, r.cols, r.x.scalar_type());
    r.vector(mean, r.rows, at::kFloat);
    r.vector(rstd, r.rows, at::kFloat);
    const Tensor dx = r.like(), dr = r.like();
    const Wgrads g(r, a[9], a[10], a[11]);
    const int64_t lddx = r.also(dx), lddr = r.also(dr);
    const double p = number(a[6]);
    const uint64_t *rng = r.rng(tensor(what, a[7])), offset = unsigned64(what, a[8]);
    call(what, [&] {
        return lm_dropout_add_layernorm_bwd(
            ptr(dy), lddy, ptr(ds), ldds, ptr(r.x), r.ld, ptr(w), ptr<float>(mean),
            ptr<float>(rstd), r.rows, r.cols, r.dtype, p, rng, offset, ptr(dx), lddx, ptr(dr),
            lddr, ptr(g.w), ptr(g.b), ptr(g.ws), g.bytes, g.flags, r.stream());
    });
    return tuple(dx, dr, g.w, g.b);
    END_HANDLE_TH_ERRORS
}

// (xs, inv_freq, positions, start, interleaved, magnitude, out, inverse) -> [y, ...]
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char* what = "lm_rope";
    count(what, n, 8);
    const bool given = a[6] != Py_None;
    // tuples, which no other thread changes meanwhile
    THPObjectPtr xs(PySequence_Tuple(a[0]));
    if (!xs) throw python_error();
    THPObjectPtr ys(given ? PySequence_Tuple(a[6]) : nullptr);
    if (given && !ys) throw python_error();
    const Py_ssize_t m = PyTuple_GET_SIZE(xs.get());
    if (m < 1 || m > 2 || (given && PyTuple_GET_SIZE(ys.get()) != m))
        refuse(what, "one or two tensors and as many outputs are wanted");
    const Tensor& x0 = tensor(what, PyTuple_GET_ITEM(xs.get(), 0));
    if (!x0.defined() || x0.dim() != 4 || !x0.is_cuda()) refuse(what, "4-D CUDA tensors are wanted");
    const at::ScalarType type = x0.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat)
        refuse(what, "bf16 or fp32 is wanted", LM_ERR_UNSUPPORTED_FORMAT);
    const int64_t batch = x0.size(0), seq = x0.size(1), dim = x0.size(3);
    const Tensor &freq = tensor(what, a[1]), &pos = tensor(what, a[2]);
    if (!freq.defined() || freq.scalar_type() != at::kDouble || freq.dim() != 1 ||
        freq.device() != x0.device() || !freq.is_contiguous())
        refuse(what, "inv_freq is a contiguous fp64 vector of the same device");
    if (pos.defined() && (pos.scalar_type() != at::kLong || pos.device() != x0.device() ||
                          pos.numel() != batch * seq || !pos.is_contiguous()))
        refuse(what, "positions is a contiguous int64 [batch, seq] of the same device");
    int overflow = 0;  // beyond 64 bits
    const long long start = PyLong_AsLongLongAndOverflow(a[3], &overflow);
    if (overflow) refuse(what, "start is a signed 64-bit integer");
    if (start == -1 && PyErr_Occurred()) throw python_error();
    const c10::cuda::OptionalCUDAGuard guard(x0.device());
    lm_rope_tensor t[2];
    Tensor y[2];
    for (Py_ssize_t i = 0; i < m; ++i) {
        const Tensor& x = tensor(what, PyTuple_GET_ITEM(xs.get(), i));
        if (!x.defined()) refuse(what, "4-D CUDA tensors are wanted");
        y[i] = given ? tensor(what, PyTuple_GET_ITEM(ys.get(), i)) : new_like(x);
        for (const Tensor* p : {&x, static_cast<const Tensor*>(&y[i])})
            if (!p->defined() || p->dim() != 4 || p->size(0) != batch || p->size(1) != seq ||
                p->size(2) != x.size(2) || p->size(3) != dim || p->scalar_type() != type ||
                p->device() != x0.device() || (dim > 1 && p->stride(3) != 1))
                refuse(what, "tensors of one type, device, batch, seq and head_dim with adjacent "
                             "elements are wanted");
        t[i] = {ptr(x),      ptr(y[i]),   x.size(2),      x.stride(0),    x.stride(1),
                x.stride(2), y[i].stride(0), y[i].stride(1), y[i].stride(2)};
    }
    const uint32_t flags =
        (truth(a[4]) ? LM_ROPE_INTERLEAVED : 0u) | (truth(a[7]) ? LM_ROPE_INVERSE : 0u);
    const float magnitude = (float)number(a[5]);
    call(what, [&] {
        return lm_rope(t, (int)m, batch, seq, dim, 2 * freq.size(0),
                       type == at::kBFloat16 ? LM_DTYPE_BF16 : LM_DTYPE_F32,
                       ptr<const double>(freq), ptr<const int64_t>(pos), start, magnitude, flags,
                       c10::cuda::getCurrentCUDAStream(x0.device().index()).stream());
    });
    PyObject* out = PyList_New(m);
    if (!out) throw python_error();
    for (Py_ssize_t i = 0; i < m; ++i) PyList_SET_ITEM(out, i, THPVariable_Wrap(y[i]));
    return out;
    END_HANDLE_TH_ERRORS
}

PyObject* use_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define CALL(f) {#f, (PyCFunction)(void*)f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(layernorm),
                         CALL(layernorm_backward),
                         CALL(dropout_add),
                         CALL(dropout_add_backward),
                         CALL(dropout_add_layernorm),
                         CALL(dropout_add_layernorm_backward),
                         CALL(rope),
                         {"use_error", use_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__native() {
    g_error = Py_NewRef(PyExc_RuntimeError);
    return PyModule_Create(&module);
}
