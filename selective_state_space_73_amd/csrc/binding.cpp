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

#include <cmath>
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

// ---------------------------------------------------------------------------
// gated delta rule

ss_head_view head_view(const Call& c, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, const char* name) {
    if (!t.is_cuda() || t.device().index() != c.idx || t.scalar_type() != type || t.sizes() != shape) c.wrong(t, shape, type, name);
    const at::IntArrayRef st = t.strides();
    if (st.back() != 1 && shape.back() > 1) refuse(PyExc_ValueError, name, ": the last dimension must be contiguous (stride 1)");
    return shape.size() == 4 ? ss_head_view{t.data_ptr(), st[0], st[1], st[2]} : ss_head_view{t.data_ptr(), st[0], 0, st[1]};
}

struct Gdr { ss_gdr_dims d; ss_gdr_args a; at::ScalarType dt; int64_t B, L, H; };

// q, k, v, g, beta, reset, scale, eps; q [B,L,k_heads,dk] and v [B,L,heads,dv], without L for one token
bool gdr_inputs(const Call& c, PyObject* const* v, PyObject* reset, PyObject* scale, PyObject* eps, bool step, Gdr* out) {
    const at::Tensor &q = tensor(v[0], "q"), &k = tensor(v[1], "k"), &x = tensor(v[2], "v");
    const int64_t n = step ? 3 : 4;
    if (q.dim() != n || x.dim() != n)
        refuse(PyExc_ValueError, step ? "q must be [streams, k_heads, dk] and v [streams, heads, dv]"
                                      : "q must be [batch, seqlen, k_heads, dk] and v [batch, seqlen, heads, dv]");
    const int64_t B = q.size(0), L = step ? 1 : q.size(1), Hk = q.size(n - 2), K = q.size(n - 1), H = x.size(n - 2), V = x.size(n - 1);
    if (Hk > INT32_MAX || H > INT32_MAX || K > INT32_MAX || V > INT32_MAX) refuse(PyExc_ValueError, "heads, dk or dv too large");
    const double sc = scale == Py_None ? 1.0 / std::sqrt((double)K) : PyFloat_AsDouble(scale);
    if (sc == -1.0 && PyErr_Occurred()) return false;
    const double ep = eps == Py_None ? 0.0 : PyFloat_AsDouble(eps);
    if (ep == -1.0 && PyErr_Occurred()) return false;
    // 0 is how the C ABI names keys that are used as they are; here that is None
    if (eps != Py_None && (float)ep == 0.0f) refuse(PyExc_ValueError, "eps must be positive in 32 bits, or None: q and k are used as they are");
    out->dt = q.scalar_type();
    out->B = B; out->L = L; out->H = H;
    out->d = ss_gdr_dims{B, L, (int32_t)Hk, (int32_t)H, (int32_t)K, (int32_t)V, io_of(out->dt, "q"), (float)sc, (float)ep, 0};
    ss_gdr_args& a = out->a;
    a = ss_gdr_args{};
    a.q = head_view(c, q, q.sizes(), out->dt, "q");
    a.k = head_view(c, k, q.sizes(), out->dt, "k");
    c10::SmallVector<int64_t, 4> shape(q.sizes().begin(), q.sizes().end() - 2);
    if (reset != Py_None) {
        const at::Tensor& t = tensor(reset, "reset");
        const auto type = t.scalar_type() == at::ScalarType::Bool ? at::ScalarType::Bool : at::ScalarType::Byte;
        a.reset = c.same<const uint8_t>(t, shape, type, "reset");
    }
    shape.push_back(H);
    a.g = c.given<float>(v[3], shape, kF32, "g");
    a.beta = c.given<float>(v[4], shape, kF32, "beta");
    shape.push_back(V);
    a.v = head_view(c, x, shape, out->dt, "v");
    return true;
}

// q, k, v, g, beta, scale, eps, state, reset, ckpt, y, workspace -> y
PyObject* gdr_fwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Call c(tensor(v[0], "q"), "q");
        Gdr x;
        if (!gdr_inputs(c, v, v[8], v[5], v[6], false, &x)) return nullptr;
        x.a.state = c.maybe<float>(v[7], {x.B, x.H, x.d.dk, x.d.dv}, kF32, "state");
        if (v[9] != Py_None) x.a.ckpt = c.given<float>(v[9], {(int64_t)ss_gdr_ckpt_floats(&x.d)}, kF32, "ckpt");
        const at::Tensor y = c.output(v[10], {x.B, x.L, x.H, x.d.dv}, x.dt, "y");
        x.a.y = y.data_ptr();
        const at::Tensor ws = c.workspace(v[11], ss_gdr_workspace_bytes(&x.d, 0));
        const ss_status s = ss_gdr_fwd(&x.d, &x.a, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, c.stream());
        return s ? status(s) : v[10] != Py_None ? Py_NewRef(v[10]) : THPVariable_Wrap(y);
    });
}

// q, k, v, g, beta, scale, eps, state, reset, y -> y
PyObject* gdr_step(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const Call c(tensor(v[0], "q"), "q");
        Gdr x;
        if (!gdr_inputs(c, v, v[8], v[5], v[6], true, &x)) return nullptr;
        if (v[7] == Py_None) refuse(PyExc_ValueError, "state is required");
        x.a.state = c.given<float>(v[7], {x.B, x.H, x.d.dk, x.d.dv}, kF32, "state");
        const at::Tensor y = c.output(v[9], {x.B, x.H, x.d.dv}, x.dt, "y");
        x.a.y = y.data_ptr();
        const ss_status s = ss_gdr_step(&x.d, &x.a, c.stream());
        return s ? status(s) : v[9] != Py_None ? Py_NewRef(v[9]) : THPVariable_Wrap(y);
    });
}

// q, k, v, g, beta, scale, eps, ckpt, dy, reset, dstate_final, workspace -> dq, dk, dv, dg, dbeta, dstate_init
PyObject* gdr_bwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Call c(tensor(v[0], "q"), "q");
        Gdr x;
        if (!gdr_inputs(c, v, v[9], v[5], v[6], false, &x)) return nullptr;
        if (v[7] == Py_None) refuse(PyExc_ValueError, "ckpt is required");
        const int64_t Hk = x.d.k_heads, K = x.d.dk, V = x.d.dv;
        x.a.ckpt = c.given<float>(v[7], {(int64_t)ss_gdr_ckpt_floats(&x.d)}, kF32, "ckpt");
        ss_gdr_grads g{};
        g.dy = c.given(v[8], {x.B, x.L, x.H, V}, x.dt, "dy");
        g.dstate_final = c.maybe<float>(v[10], {x.B, x.H, K, V}, kF32, "dstate_final");
        const at::Tensor dq = c.empty({x.B, x.L, Hk, K}, x.dt), dk = c.empty({x.B, x.L, Hk, K}, x.dt);
        const at::Tensor dv = c.empty({x.B, x.L, x.H, V}, x.dt), dg = c.empty({x.B, x.L, x.H}, kF32), db = c.empty({x.B, x.L, x.H}, kF32);
        const at::Tensor dh = c.empty({x.B, x.H, K, V}, kF32);
        g.dq = dq.data_ptr(); g.dk = dk.data_ptr(); g.dv = dv.data_ptr();
        g.dg = static_cast<float*>(dg.data_ptr());
        g.dbeta = static_cast<float*>(db.data_ptr());
        g.dstate_init = static_cast<float*>(dh.data_ptr());
        const at::Tensor ws = c.workspace(v[11], ss_gdr_workspace_bytes(&x.d, 1));
        const ss_status s = ss_gdr_bwd(&x.d, &x.a, &g, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, c.stream());
        return s ? status(s) : results(dq, dk, dv, dg, db, dh);
    });
}

// ---------------------------------------------------------------------------
// the norms around a layer

struct Gnorm { ss_gnorm_dims d; ss_gnorm_args a; at::ScalarType dt; };

// y, w, gate, residual, scale, w_next, eps
bool gnorm_inputs(const Call& c, PyObject* const* v, Gnorm* out) {
    const at::Tensor &y = tensor(v[0], "y"), &w = tensor(v[1], "w");
    const Rows r = rows_of(y, "y");
    const double eps = PyFloat_AsDouble(v[6]);
    if (eps == -1.0 && PyErr_Occurred()) return false;
    if (w.dim() != 1) refuse(PyExc_ValueError, "w must be [group]");
    out->dt = y.scalar_type();
    out->d = ss_gnorm_dims{r.M, r.K, w.size(0), io_of(out->dt, "y"), (float)eps};
    ss_gnorm_args& a = out->a;
    a = ss_gnorm_args{};
    a.y = y.data_ptr();
    a.w = c.same<float>(w, {w.size(0)}, kF32, "w");
    a.gate = c.maybe(v[2], y.sizes(), out->dt, "gate");
    a.residual = c.maybe(v[3], y.sizes(), out->dt, "residual");
    a.scale = c.maybe<float>(v[4], {r.K}, kF32, "scale");
    a.w_next = c.maybe<float>(v[5], {r.K}, kF32, "w_next");
    return true;
}

// y, w, gate, residual, scale, w_next, eps, s, n -> s, n
PyObject* gnorm_fwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor& y = tensor(v[0], "y");
        const Call c(y, "y");
        Gnorm x;
        if (!gnorm_inputs(c, v, &x)) return nullptr;
        if (v[5] == Py_None && v[8] != Py_None) refuse(PyExc_ValueError, "n given without w_next");
        const at::Tensor s = c.output(v[7], y.sizes(), x.dt, "s");
        at::Tensor m;
        if (v[5] != Py_None) m = c.output(v[8], y.sizes(), x.dt, "n");
        x.a.s = s.data_ptr();
        x.a.n = m.defined() ? m.data_ptr() : nullptr;
        const ss_status e = ss_gnorm_fwd(&x.d, &x.a, c.stream());
        return e ? status(e) : results(s, m);
    });
}

// y, w, gate, residual, scale, w_next, eps, ds, dn, workspace -> dy, dw, dgate, dresidual, dscale, dw_next
PyObject* gnorm_bwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const at::Tensor& y = tensor(v[0], "y");
        const Call c(y, "y");
        Gnorm x;
        if (!gnorm_inputs(c, v, &x)) return nullptr;
        ss_gnorm_grads g{};
        g.ds = c.maybe(v[7], y.sizes(), x.dt, "ds");
        g.dn = c.maybe(v[8], y.sizes(), x.dt, "dn");
        const at::Tensor dy = c.empty(y.sizes(), x.dt), dw = c.empty({x.d.group}, kF32);
        at::Tensor dz, dr, da, dm;
        if (x.a.gate) dz = c.empty(y.sizes(), x.dt);
        if (x.a.residual) dr = c.empty(y.sizes(), x.dt);
        if (x.a.scale) da = c.empty({x.d.cols}, kF32);
        if (x.a.w_next) dm = c.empty({x.d.cols}, kF32);
        auto at_of = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
        g.dy = dy.data_ptr(); g.dgate = at_of(dz); g.dresidual = at_of(dr);
        g.dw = static_cast<float*>(dw.data_ptr());
        g.dscale = static_cast<float*>(at_of(da));
        g.dw_next = static_cast<float*>(at_of(dm));
        const at::Tensor ws = c.workspace(v[9], ss_gnorm_workspace_bytes(&x.d));
        const ss_status e = ss_gnorm_bwd(&x.d, &x.a, &g, at_of(ws), ws.defined() ? ws.nbytes() : 0, c.stream());
        return e ? status(e) : results(dy, dw, dz, dr, da, dm);
    });
}

#define FN(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FN(glr_fwd), FN(glr_step), FN(glr_bwd), FN(quant), FN(norm), FN(gemm), FN(gdr_fwd), FN(gdr_step),
                           FN(gdr_bwd), FN(gnorm_fwd), FN(gnorm_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
