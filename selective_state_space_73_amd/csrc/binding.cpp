// Python binding of the operators around the scan, as a C extension: checks of the tensors,
// outputs and workspaces from torch's allocator, torch's current stream, one call of the C ABI.
//
// A decode step waits for what a call costs on the host before its kernel starts, so the
// small calls' time is this file's: with the same steps in Python (ctypes) a call of
// ss_glr_step took 8.7 us of host time, of which the launch is 3.
//
// Each function takes its operands by position (None where one is absent) and returns its
// results, or the C ABI's status as an int where the call was refused; the Python wrappers hold
// names, defaults and documentation. Wrong dtypes raise TypeError, wrong devices, shapes and
// layouts ValueError. No C++ exception leaves a function.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>

#include "selscan_ops.h"

namespace {

constexpr int64_t kBlock = 128;
constexpr auto kQ8 = at::ScalarType::Float8_e4m3fn;
constexpr auto kF32 = at::ScalarType::Float;

struct Refusal { PyObject* type; std::string text; };

template <typename... P>
[[noreturn]] void refuse(PyObject* type, const P&... parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw Refusal{type, s.str()};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// The tensors of one call are on one GPU; the call runs there, whichever is current.
struct Call {
    int idx;
    c10::DeviceGuard guard;
    explicit Call(const at::Tensor& x, const char* name) : idx(device_of(x, name)), guard(x.device()) {}
    static int device_of(const at::Tensor& x, const char* name) {
        if (!x.is_cuda()) refuse(PyExc_ValueError, name, " must be a device tensor, got ", x.device());
        return x.device().index();
    }
    void* stream() const { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)idx).stream(); }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
        return at::empty(shape, at::TensorOptions().dtype(t).device(at::DeviceType::CUDA, (c10::DeviceIndex)idx));
    }

    [[noreturn]] void wrong(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, const char* name) const {
        if (!t.is_cuda() || t.device().index() != idx)
            refuse(PyExc_ValueError, name, " must be on cuda:", idx, ", got ", t.device());
        if (t.scalar_type() != type) refuse(PyExc_TypeError, name, " must be ", type, ", got ", t.scalar_type());
        refuse(PyExc_ValueError, name, " has shape ", t.sizes(), ", expected ", shape, ", contiguous");
    }
    // the data pointer of a contiguous tensor of this shape, dtype and device
    template <typename T = void>
    T* same(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, const char* name) const {
        if (!t.is_cuda() || t.device().index() != idx || t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
            wrong(t, shape, type, name);
        return static_cast<T*>(t.data_ptr());
    }
    template <typename T = void>
    T* given(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const char* name) const {
        return same<T>(tensor(o, name), shape, type, name);
    }
    template <typename T = void>
    T* maybe(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const char* name) const {
        return o == Py_None ? nullptr : given<T>(o, shape, type, name);
    }
    // an output: the caller's, or a new one
    at::Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const char* name) const {
        if (o == Py_None) return empty(shape, type);
        given(o, shape, type, name);
        return THPVariable_Unpack(o);
    }
    ss_view view(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const char* name) const {
        const at::Tensor& t = tensor(o, name);
        if (!t.is_cuda() || t.device().index() != idx || t.scalar_type() != type || t.sizes() != shape) wrong(t, shape, type, name);
        const at::IntArrayRef st = t.strides();
        if (st.back() != 1 && shape.back() > 1) refuse(PyExc_ValueError, name, ": channels must be contiguous (last stride 1)");
        return ss_view{t.data_ptr(), st[0], st[1]};
    }
    at::Tensor workspace(PyObject* o, size_t need) const {
        if (o == Py_None) return need ? empty({(int64_t)need}, at::ScalarType::Byte) : at::Tensor();
        const at::Tensor& t = tensor(o, "workspace");
        if (!t.is_cuda() || t.device().index() != idx) refuse(PyExc_ValueError, "workspace must be on cuda:", idx);
        if (!t.is_contiguous() || t.nbytes() < need)
            refuse(PyExc_ValueError, "workspace must be contiguous, of at least ", need, " bytes");
        return t;
    }
};

int io_of(at::ScalarType t, const char* name) {
    if (t == at::ScalarType::BFloat16) return SS_BF16;
    if (t == kF32) return SS_F32;
    refuse(PyExc_TypeError, name, " must be float32 or bfloat16, got ", t);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
    try {
        if (n != want) refuse(PyExc_TypeError, "expected ", want, " arguments, got ", n);
        return f();
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (...) {                                        // torch's own, the allocator's out of memory among them
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

PyObject* status(ss_status s) { return PyLong_FromLong((long)s); }

template <typename... T>
PyObject* results(const T&... t) {
    PyObject* out = PyTuple_New(sizeof...(t));
    if (!out) return nullptr;
    Py_ssize_t k = 0;
    bool ok = true;
    auto put = [&](const at::Tensor& v) {
        PyObject* o = v.defined() ? THPVariable_Wrap(v) : Py_NewRef(Py_None);
        ok = ok && o;
        PyTuple_SET_ITEM(out, k++, o);
    };
    (put(t), ...);
    if (!ok) { Py_DECREF(out); return nullptr; }
    return out;
}

// ---------------------------------------------------------------------------
// gated linear recurrence

ss_glr_args glr_args(const Call& c, PyObject* x, PyObject* r, PyObject* i, PyObject* A, PyObject* reset, at::IntArrayRef shape,
                     at::ScalarType dt) {
    ss_glr_args a{};
    a.x = c.view(x, shape, dt, "x");
    a.r = c.view(r, shape, dt, "r");
    a.i = c.view(i, shape, dt, "i");
    a.A = c.given<float>(A, {shape.back()}, kF32, "A");
    if (reset != Py_None) {
        const at::Tensor& t = tensor(reset, "reset");
        const auto type = t.scalar_type() == at::ScalarType::Bool ? at::ScalarType::Bool : at::ScalarType::Byte;
        a.reset = c.same<const uint8_t>(t, shape.slice(0, shape.size() - 1), type, "reset");
    }
    return a;
}

// x, r, i, A, state, reset, ckpt, y, workspace -> y
PyObject* glr_fwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor& x = tensor(v[0], "x");
        const Call c(x, "x");
        if (x.dim() != 3) refuse(PyExc_ValueError, "x must be [batch, seqlen, d]");
        const at::IntArrayRef shape = x.sizes();
        const int64_t B = shape[0], L = shape[1], D = shape[2], K = (L + SS_GLR_CKPT - 1) / SS_GLR_CKPT;
        const auto dt = x.scalar_type();
        const ss_glr_dims d{B, L, D, io_of(dt, "x"), 0};
        ss_glr_args a = glr_args(c, v[0], v[1], v[2], v[3], v[5], shape, dt);
        a.state = c.maybe<float>(v[4], {B, D}, kF32, "state");
        a.ckpt = c.maybe<float>(v[6], {B, K, D}, kF32, "ckpt");
        const at::Tensor y = c.output(v[7], shape, dt, "y");
        a.y = y.data_ptr();
        const at::Tensor ws = c.workspace(v[8], ss_glr_workspace_bytes(&d, 0));
        const ss_status s = ss_glr_fwd(&d, &a, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, c.stream());
        return s ? status(s) : v[7] != Py_None ? Py_NewRef(v[7]) : THPVariable_Wrap(y);
    });
}

// x, r, i, A, state, reset, y -> y
PyObject* glr_step(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor& x = tensor(v[0], "x");
        const Call c(x, "x");
        if (x.dim() != 2) refuse(PyExc_ValueError, "x must be [streams, d]");
        if (v[4] == Py_None) refuse(PyExc_ValueError, "state is required");
        const at::IntArrayRef shape = x.sizes();
        const auto dt = x.scalar_type();
        const ss_glr_dims d{shape[0], 1, shape[1], io_of(dt, "x"), 0};
        ss_glr_args a = glr_args(c, v[0], v[1], v[2], v[3], v[5], shape, dt);
        a.state = c.given<float>(v[4], shape, kF32, "state");
        const at::Tensor y = c.output(v[6], shape, dt, "y");
        a.y = y.data_ptr();
        const ss_status s = ss_glr_step(&d, &a, c.stream());
        return s ? status(s) : v[6] != Py_None ? Py_NewRef(v[6]) : THPVariable_Wrap(y);
    });
}

// x, r, i, A, ckpt, dy, reset, dstate_final, workspace -> dx, dr, di, dA, dstate_init
PyObject* glr_bwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor& x = tensor(v[0], "x");
        const Call c(x, "x");
        if (x.dim() != 3) refuse(PyExc_ValueError, "x must be [batch, seqlen, d]");
        if (v[4] == Py_None) refuse(PyExc_ValueError, "ckpt is required");
        const at::IntArrayRef shape = x.sizes();
        const int64_t B = shape[0], L = shape[1], D = shape[2], K = (L + SS_GLR_CKPT - 1) / SS_GLR_CKPT;
        const auto dt = x.scalar_type();
        const ss_glr_dims d{B, L, D, io_of(dt, "x"), 0};
        ss_glr_args a = glr_args(c, v[0], v[1], v[2], v[3], v[6], shape, dt);
        a.ckpt = c.given<float>(v[4], {B, K, D}, kF32, "ckpt");
        ss_glr_grads g{};
        g.dy = c.given(v[5], shape, dt, "dy");
        g.dstate_final = c.maybe<float>(v[7], {B, D}, kF32, "dstate_final");
        const at::Tensor dx = c.empty(shape, dt), dr = c.empty(shape, dt), di = c.empty(shape, dt);
        const at::Tensor dA = c.empty({D}, kF32), dh = c.empty({B, D}, kF32);
        g.dx = dx.data_ptr(); g.dr = dr.data_ptr(); g.di = di.data_ptr();
        g.dA = static_cast<float*>(dA.data_ptr());
        g.dstate_init = static_cast<float*>(dh.data_ptr());
        const at::Tensor ws = c.workspace(v[8], ss_glr_workspace_bytes(&d, 1));
        const ss_status s = ss_glr_bwd(&d, &a, &g, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, c.stream());
        return s ? status(s) : results(dx, dr, di, dA, dh);
    });
}

// ---------------------------------------------------------------------------
// 8-bit floating point with block scales

struct Rows { int64_t M, K, KB; c10::SmallVector<int64_t, 6> scales; };     // of a contiguous [..., K]

Rows rows_of(const at::Tensor& x, const char* name) {
    if (x.dim() < 1 || !x.is_contiguous())
        refuse(PyExc_ValueError, name, " must be contiguous, with at least one dimension");
    Rows r;
    r.K = x.sizes().back();
    r.M = r.K ? x.numel() / r.K : 0;
    r.KB = (r.K + kBlock - 1) / kBlock;
    r.scales.assign(x.sizes().begin(), x.sizes().end());
    r.scales.back() = r.KB;
    return r;
}

// x, square, q, scale -> q, scale
PyObject* quant(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        const at::Tensor& x = tensor(v[0], "x");
        const Call c(x, "x");
        Rows r = rows_of(x, "x");
        const int square = PyObject_IsTrue(v[1]);
        if (square < 0) return nullptr;
        if (square && x.dim() != 2) refuse(PyExc_ValueError, "a square rounding takes x [N, K]");
        if (square) r.scales[0] = (r.M + kBlock - 1) / kBlock;
        const ss_q8_dims d{r.M, r.K, io_of(x.scalar_type(), "x"), square, 0.0f, 0};
        const at::Tensor q = c.output(v[2], x.sizes(), kQ8, "q"), scale = c.output(v[3], r.scales, kF32, "scale");
        const ss_status s = ss_quant_q8(&d, x.data_ptr(), q.data_ptr(), static_cast<float*>(scale.data_ptr()), c.stream());
        return s ? status(s) : results(q, scale);
    });
}

// x, w, residual, eps, q, scale, sum_out -> q, scale, sum
PyObject* norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor& x = tensor(v[0], "x");
        const Call c(x, "x");
        const Rows r = rows_of(x, "x");
        const auto dt = x.scalar_type();
        const double eps = PyFloat_AsDouble(v[3]);
        if (eps == -1.0 && PyErr_Occurred()) return nullptr;
        if (v[2] == Py_None && v[6] != Py_None) refuse(PyExc_ValueError, "sum_out given without a residual");
        const ss_q8_dims d{r.M, r.K, io_of(dt, "x"), 0, (float)eps, 0};
        ss_norm_q8_args a{};
        a.x = x.data_ptr();
        a.residual = c.maybe(v[2], x.sizes(), dt, "residual");
        a.w = c.given<float>(v[1], {r.K}, kF32, "w");
        const at::Tensor q = c.output(v[4], x.sizes(), kQ8, "q"), scale = c.output(v[5], r.scales, kF32, "scale");
        at::Tensor sum;
        if (v[2] != Py_None) sum = c.output(v[6], x.sizes(), dt, "sum_out");
        a.q = q.data_ptr();
        a.scale = static_cast<float*>(scale.data_ptr());
        a.sum = sum.defined() ? sum.data_ptr() : nullptr;
        const ss_status s = ss_norm_q8(&d, &a, c.stream());
        return s ? status(s) : results(q, scale, sum);
    });
}

// xq, xs, wq, ws, residual, out, out_dtype -> y
PyObject* gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor &xq = tensor(v[0], "xq"), &wq = tensor(v[2], "wq");
        const Call c(xq, "xq");
        Rows r = rows_of(xq, "xq");
        if (wq.dim() != 2) refuse(PyExc_ValueError, "wq must be [N, K]");
        const int64_t N = wq.size(0);
        if (v[5] == Py_None && !THPDtype_Check(v[6])) refuse(PyExc_TypeError, "out_dtype must be a torch.dtype");
        const auto dt = v[5] != Py_None ? tensor(v[5], "out").scalar_type() : reinterpret_cast<THPDtype*>(v[6])->scalar_type;
        const ss_gemm_q8_dims d{r.M, N, r.K, io_of(dt, "out"), 0};
        ss_gemm_q8_args a{};
        a.xq = c.same(xq, xq.sizes(), kQ8, "xq");
        a.xs = c.given<float>(v[1], r.scales, kF32, "xs");
        a.wq = c.same(wq, {N, r.K}, kQ8, "wq");
        a.ws = c.given<float>(v[3], {(N + kBlock - 1) / kBlock, r.KB}, kF32, "ws");
        r.scales.back() = N;                              // from here on y's shape
        a.residual = c.maybe(v[4], r.scales, dt, "residual");
        const at::Tensor y = c.output(v[5], r.scales, dt, "out");
        a.y = y.data_ptr();
        const ss_status s = ss_gemm_q8(&d, &a, c.stream());
        return s ? status(s) : v[5] != Py_None ? Py_NewRef(v[5]) : THPVariable_Wrap(y);
    });
}

#define FN(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FN(glr_fwd), FN(glr_step), FN(glr_bwd), FN(quant), FN(norm), FN(gemm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
