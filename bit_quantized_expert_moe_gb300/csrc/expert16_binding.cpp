// Python binding of the 16-bit expert operators: argument marshalling only.
//
// A small call takes a few microseconds on the GPU; checking shapes, taking
// pointers and making outputs in the interpreter takes longer than that on the
// GPU's host (swiglu of 8 rows: 7.3 us a call there, 3.7 here; the gradients of
// a block norm: 20 and 9).  Shapes and types are checked here, everything else
// by the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <exception>
#include <functional>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "moe_w4.h"

namespace {

using at::Tensor;
using Shape = at::IntArrayRef;

PyObject* g_check = nullptr;  // raises MoeError(status, what)

// A ValueError on its way out.
struct Refusal : std::runtime_error {
    using std::runtime_error::runtime_error;
};
// A Python error that is already set.
struct Raised {};

std::string text(Shape s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}
[[noreturn]] void refuse(const char* what, const Tensor& t, Shape shape, at::ScalarType type) {
    throw Refusal(std::string(what) + ": shape " + text(shape) + " of " + at::toString(type) + " expected, not " +
                  text(t.sizes()) + " of " + at::toString(t.scalar_type()));
}
void want(const char* what, const Tensor& t, Shape shape, at::ScalarType type) {
    if (t.scalar_type() != type || t.sizes() != shape) refuse(what, t, shape, type);
}

moe_dtype_t moe_type(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return MOE_DT_BF16;
        case at::kHalf: return MOE_DT_F16;
        case at::kFloat: return MOE_DT_F32;
        default: throw Refusal(std::string("bfloat16, float16 or float32 tensor expected, not ") + at::toString(t));
    }
}

// The tensors of a call that are there: dense, and on the device of the first, on
// which the call runs.  Where autograd records, it learns nothing of the call: said
// once for each place of a program (as the warnings' filters have it).
void on_one_device(std::initializer_list<std::reference_wrapper<const Tensor>> ts) {
    const Tensor& first = *ts.begin();
    for (const Tensor& t : ts)
        if (t.defined() && t.requires_grad() && at::GradMode::is_enabled()) {
            if (PyErr_WarnEx(PyExc_UserWarning,
                             "an operand requires gradients, but the 16-bit expert operators record no graph: their outputs "
                             "do not require gradients; call them under torch.no_grad() and take the gradients from "
                             "grouped_mm_dx, grouped_mm_dw, swiglu_backward and block_norm_backward", 1) < 0)
                throw Raised{};
            break;
        }
    for (const Tensor& t : ts) {
        if (!t.defined()) continue;
        if (!t.is_cuda()) throw Refusal("device tensor expected");
        if (!t.is_contiguous()) throw Refusal("contiguous tensor expected");
        if (t.device() != first.device())
            throw Refusal("tensors of one device expected, not of " + first.device().str() + " and " + t.device().str());
    }
}
// Pointer of a tensor that on_one_device() has seen, null for one that is not there.
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <class T>
T* ptr_as(const Tensor& t) { return static_cast<T*>(ptr(t)); }

// Arguments of a call by position or name, in the order of `names`; the first
// `needed` have to be there.
template <size_t N>
struct Args {
    std::array<PyObject*, N> v{};
    Args(const char* fn, const std::array<PyObject*, N>& names, size_t needed, PyObject* const* args, Py_ssize_t n,
         PyObject* kw) {
        if (n > (Py_ssize_t)N) throw_type(std::string(fn) + "() takes at most " + std::to_string(N) + " arguments");
        for (Py_ssize_t i = 0; i < n; ++i) v[i] = args[i];
        const Py_ssize_t k = kw ? PyTuple_GET_SIZE(kw) : 0;
        for (Py_ssize_t i = 0; i < k; ++i) {
            PyObject* name = PyTuple_GET_ITEM(kw, i);
            size_t at = 0;
            while (at < N && names[at] != name) ++at;
            if (at == N)
                for (at = 0; at < N && PyUnicode_Compare(names[at], name) != 0;) ++at;
            if (at == N) throw_type(std::string(fn) + "() got an unexpected argument '" + utf8(name) + "'");
            if (v[at]) throw_type(std::string(fn) + "() got two values for argument '" + utf8(name) + "'");
            v[at] = args[n + i];
        }
        for (size_t i = 0; i < needed; ++i)
            if (!v[i]) throw_type(std::string(fn) + "() misses argument '" + utf8(names[i]) + "'");
    }
    static std::string utf8(PyObject* s) {
        const char* c = PyUnicode_AsUTF8(s);
        return c ? c : "?";
    }
    [[noreturn]] static void throw_type(const std::string& s) {
        PyErr_SetString(PyExc_TypeError, s.c_str());
        throw Raised{};
    }
    bool given(size_t i) const { return v[i] && v[i] != Py_None; }
    // Undefined where there is none.
    Tensor tensor(size_t i) const {
        if (!given(i)) return Tensor();
        if (!THPVariable_Check(v[i])) throw_type("tensor expected");
        return THPVariable_Unpack(v[i]);
    }
    Tensor needed_tensor(size_t i) const {
        if (!given(i)) throw_type("tensor expected");
        return tensor(i);
    }
    float number(size_t i, double otherwise) const {
        if (!v[i]) return (float)otherwise;
        const double d = PyFloat_AsDouble(v[i]);
        if (d == -1.0 && PyErr_Occurred()) throw Raised{};
        return (float)d;
    }
};

// The device of `of` and the stream of a call there: the one given, else that
// device's current one.  While this lives both are current, so that the call launches
// on that device and what it allocates belongs to the stream that writes it.
struct OnStream {
    cudaStream_t s;
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard guard;
    template <size_t N>
    OnStream(const Args<N>& a, size_t i, const Tensor& of) {
        const c10::DeviceIndex index = of.device().index();
        if (c10::cuda::current_device() != index) device.set_index(index);
        if (!a.given(i)) {
            s = c10::cuda::getCurrentCUDAStream(index).stream();
            return;
        }
        PyObject* h = PyObject_GetAttrString(a.v[i], "cuda_stream");
        if (!h) throw Raised{};
        s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
        Py_DECREF(h);
        if (!s && PyErr_Occurred()) throw Raised{};
        guard.reset_stream(c10::cuda::getStreamFromExternal(s, index));
    }
};

// Interned argument names, made once.
template <size_t N>
std::array<PyObject*, N> intern(const std::array<const char*, N>& s) {
    std::array<PyObject*, N> r;
    for (size_t i = 0; i < N; ++i) r[i] = PyUnicode_InternFromString(s[i]);
    return r;
}

void check(moe_status_t st, const char* what) {
    if (st == MOE_OK) return;
    PyObject* r = PyObject_CallFunction(g_check, "is", (int)st, what);
    Py_XDECREF(r);
    if (r) PyErr_SetString(PyExc_RuntimeError, what);  // not reached: the call raises
    throw Raised{};
}

// Runs a body that may throw; no C++ exception leaves for the interpreter.
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Raised&) {
    } catch (const Refusal& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        // torch.OutOfMemoryError, as from torch's own functions (its C++ name is not exported)
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// A new tensor beside `like`, or the one given, of that shape and type.
Tensor output(const Tensor& given, const char* what, const Tensor& like, Shape shape, at::ScalarType type) {
    if (given.defined()) {
        want(what, given, shape, type);
        return given;
    }
    // Straight from the CUDA allocator: 0.3 us less per output than at::empty's
    // dispatch, of the 3.8 us that the smallest call takes.
    return at::detail::empty_cuda(shape, type, like.device(), c10::nullopt);
}
// The workspace given, or a new one; `like` as for output().
Tensor workspace(const Tensor& given, size_t bytes, const Tensor& like) {
    return given.defined() ? given : output(given, "ws", like, {(int64_t)std::max<size_t>(bytes, 256)}, at::kByte);
}
PyObject* wrap(const Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <size_t N>
PyObject* wrap_all(const Tensor (&ts)[N]) {
    PyObject* r = PyTuple_New(N);
    if (!r) throw Raised{};
    for (size_t i = 0; i < N; ++i) {
        PyObject* o = wrap(ts[i]);
        if (!o) {
            Py_DECREF(r);
            throw Raised{};
        }
        PyTuple_SET_ITEM(r, i, o);
    }
    return r;
}
int32_t size32(int64_t v) {
    if (v > INT32_MAX) throw Refusal("a size is beyond 32 bits");
    return (int32_t)v;
}
void dims(const char* what, const Tensor& t, int64_t n) {
    if (t.dim() != n) throw Refusal(std::string(what) + ": " + std::to_string(n) + " dimensions expected, not " + text(t.sizes()));
}

// ------------------------------------------------------------ grouped products
using GroupedFn = moe_status_t (*)(moe_dtype_t, const void*, const void*, const int32_t*, int32_t, int32_t, int32_t,
                                   int32_t, void*, void*, size_t, cudaStream_t);

PyObject* grouped(GroupedFn fn, const char* name, const Tensor& a, const Tensor& b, const Tensor& offsets, int64_t R,
                  int64_t E, int64_t N, int64_t K, const Tensor& out, const Tensor& given_ws, cudaStream_t s) {
    want("offsets", offsets, {E + 1}, at::kInt);
    const int32_t r = size32(R), e = size32(E), n = size32(N), k = size32(K);
    const moe_dtype_t dt = moe_type(a.scalar_type());
    const Tensor ws = workspace(given_ws, given_ws.defined() ? 0 : moe_grouped_mm_workspace_size(r, e, n, k), offsets);
    check(fn(dt, ptr(a), ptr(b), ptr_as<int32_t>(offsets), r, e, n, k, ptr(out), ptr(ws), (size_t)ws.numel(), s), name);
    return wrap(out);
}

PyObject* py_grouped_mm(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    return guarded([&] {
        static const auto names = intern<6>({"x", "w", "offsets", "y", "ws", "stream"});
        const Args<6> a("grouped_mm", names, 3, args, n, kw);
        const Tensor x = a.needed_tensor(0), w = a.needed_tensor(1), off = a.needed_tensor(2);
        dims("x", x, 2);
        dims("w", w, 3);
        const int64_t R = x.size(0), K = x.size(1), E = w.size(0), N = w.size(1);
        want("w", w, {E, N, K}, x.scalar_type());
        const Tensor given = a.tensor(3), ws = a.tensor(4);
        on_one_device({x, w, off, given, ws});
        const OnStream on(a, 5, x);
        const Tensor y = output(given, "y", x, {R, N}, x.scalar_type());
        return grouped(moe_grouped_mm, "moe_grouped_mm", x, w, off, R, E, N, K, y, ws, on.s);
    });
}
PyObject* py_grouped_mm_dx(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    return guarded([&] {
        static const auto names = intern<6>({"dy", "w", "offsets", "dx", "ws", "stream"});
        const Args<6> a("grouped_mm_dx", names, 3, args, n, kw);
        const Tensor dy = a.needed_tensor(0), w = a.needed_tensor(1), off = a.needed_tensor(2);
        dims("dy", dy, 2);
        dims("w", w, 3);
        const int64_t R = dy.size(0), N = dy.size(1), E = w.size(0), K = w.size(2);
        want("w", w, {E, N, K}, dy.scalar_type());
        const Tensor given = a.tensor(3), ws = a.tensor(4);
        on_one_device({dy, w, off, given, ws});
        const OnStream on(a, 5, dy);
        const Tensor dx = output(given, "dx", dy, {R, K}, dy.scalar_type());
        return grouped(moe_grouped_mm_dx, "moe_grouped_mm_dx", dy, w, off, R, E, N, K, dx, ws, on.s);
    });
}
PyObject* py_grouped_mm_dw(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    return guarded([&] {
        static const auto names = intern<6>({"dy", "x", "offsets", "dw", "ws", "stream"});
        const Args<6> a("grouped_mm_dw", names, 3, args, n, kw);
        const Tensor dy = a.needed_tensor(0), x = a.needed_tensor(1), off = a.needed_tensor(2);
        dims("dy", dy, 2);
        dims("x", x, 2);
        const int64_t R = dy.size(0), N = dy.size(1), K = x.size(1), E = off.numel() - 1;
        want("x", x, {R, K}, dy.scalar_type());
        const Tensor given = a.tensor(3), ws = a.tensor(4);
        on_one_device({dy, x, off, given, ws});
        const OnStream on(a, 5, dy);
        const Tensor dw = output(given, "dw", dy, {E, N, K}, dy.scalar_type());
        return grouped(moe_grouped_mm_dw, "moe_grouped_mm_dw", dy, x, off, R, E, N, K, dw, ws, on.s);
    });
}

// ------------------------------------------------------------ gated activation
int64_t gated_width(const Tensor& gu, const Tensor& row_w, const Tensor& row_map) {
    dims("gu", gu, 2);
    const int64_t R = gu.size(0), F2 = gu.size(1);
    if (F2 & 1) throw Refusal("gu holds the gate and the up half of every row");
    if (row_w.defined()) want("row_w", row_w, {R}, at::kFloat);
    if (row_map.defined()) want("row_map", row_map, {R}, at::kInt);
    return F2 >> 1;
}
PyObject* py_swiglu(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    return guarded([&] {
        static const auto names = intern<5>({"gu", "row_w", "row_map", "h", "stream"});
        const Args<5> a("swiglu", names, 1, args, n, kw);
        const Tensor gu = a.needed_tensor(0), row_w = a.tensor(1), row_map = a.tensor(2);
        const int64_t F = gated_width(gu, row_w, row_map), R = gu.size(0);
        const moe_dtype_t dt = moe_type(gu.scalar_type());
        const Tensor given = a.tensor(3);
        on_one_device({gu, row_w, row_map, given});
        const OnStream on(a, 4, gu);
        const Tensor h = output(given, "h", gu, {R, F}, gu.scalar_type());
        check(moe_swiglu(dt, ptr(gu), ptr_as<float>(row_w), ptr_as<int32_t>(row_map), size32(R), size32(F), ptr(h),
                         on.s), "moe_swiglu");
        return wrap(h);
    });
}
PyObject* py_swiglu_backward(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    return guarded([&] {
        static const auto names = intern<7>({"dh", "gu", "row_w", "row_map", "dgu", "drow_w", "stream"});
        const Args<7> a("swiglu_backward", names, 2, args, n, kw);
        const Tensor dh = a.needed_tensor(0), gu = a.needed_tensor(1), row_w = a.tensor(2), row_map = a.tensor(3);
        const int64_t F = gated_width(gu, row_w, row_map), R = gu.size(0);
        const at::ScalarType t = gu.scalar_type();
        const moe_dtype_t dt = moe_type(t);
        want("dh", dh, {R, F}, t);
        const Tensor given = a.tensor(4);
        Tensor dw = a.tensor(5);
        on_one_device({gu, dh, row_w, row_map, given, dw});
        const OnStream on(a, 6, gu);
        const Tensor dgu = output(given, "dgu", gu, {R, 2 * F}, t);
        if (dw.defined() || row_w.defined()) dw = output(dw, "drow_w", gu, {R}, at::kFloat);
        check(moe_swiglu_backward(dt, ptr(dh), ptr(gu), ptr_as<float>(row_w), ptr_as<int32_t>(row_map), size32(R),
                                  size32(F), ptr(dgu), ptr_as<float>(dw), on.s), "moe_swiglu_backward");
        return wrap_all({dgu, dw});
    });
}

// ----------------------------------------------------------------- block norms
struct Norm {
    int64_t T, D, G = 1;
    moe_dtype_t dt, pt;
    at::ScalarType type, ptype;
    Norm(const Tensor& x, const Tensor& post, const Tensor& gate, const Tensor& pre) {
        dims("x", x, 2);
        T = x.size(0);
        D = x.size(1);
        type = x.scalar_type();
        dt = moe_type(type);
        ptype = gate.defined() ? gate.scalar_type() : post.defined() ? post.scalar_type() : pre.defined() ? pre.scalar_type() : type;
        pt = moe_type(ptype);
        if (gate.defined()) {
            G = gate.dim() == 2 ? gate.size(0) : 0;
            if (G < 1 || T % G || gate.size(1) != D)
                throw Refusal("gate: [G, " + std::to_string(D) + "] with G a divisor of " + std::to_string(T) +
                              " rows expected, not " + text(gate.sizes()));
        }
        if (post.defined()) want("gamma_post", post, {D}, ptype);
        if (pre.defined()) want("gamma_pre", pre, {D}, ptype);
    }
    void row(const char* what, const Tensor& t) const {
        if (t.defined()) want(what, t, {T, D}, type);
    }
};

PyObject* py_block_norm(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    return guarded([&] {
        static const auto names = intern<10>({"x", "y", "gamma_post", "gate", "gamma_pre", "alpha", "eps", "x_out", "h", "stream"});
        const Args<10> a("block_norm", names, 1, args, n, kw);
        const Tensor x = a.needed_tensor(0), y = a.tensor(1), post = a.tensor(2), gate = a.tensor(3), pre = a.tensor(4);
        const Norm m(x, post, gate, pre);
        m.row("y", y);
        Tensor xo = a.tensor(7), h = a.tensor(8);
        on_one_device({x, y, post, gate, pre, xo, h});
        const OnStream on(a, 9, x);
        if (xo.defined() || y.defined()) xo = output(xo, "x_out", x, {m.T, m.D}, m.type);
        if (h.defined() || pre.defined()) h = output(h, "h", x, {m.T, m.D}, m.type);
        check(moe_block_norm(m.dt, m.pt, size32(m.T), size32(m.D), size32(m.G), a.number(5, 1.0), a.number(6, 1e-6),
                             ptr(post), ptr(gate), ptr(pre), ptr(x), ptr(y), ptr(xo), ptr(h), on.s), "moe_block_norm");
        return wrap_all({xo, h});
    });
}
PyObject* py_block_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    return guarded([&] {
        static const auto names = intern<11>({"x_out", "y", "dx_out", "dh", "gamma_post", "gate", "gamma_pre", "alpha",
                                              "eps", "ws", "stream"});
        const Args<11> a("block_norm_backward", names, 1, args, n, kw);
        const Tensor x = a.needed_tensor(0), y = a.tensor(1), dxo = a.tensor(2), dh = a.tensor(3);
        const Tensor post = a.tensor(4), gate = a.tensor(5), pre = a.tensor(6), given_ws = a.tensor(9);
        const Norm m(x, post, gate, pre);
        m.row("y", y);
        m.row("dx_out", dxo);
        m.row("dh", dh);
        const int32_t T = size32(m.T), D = size32(m.D), G = size32(m.G);
        on_one_device({x, y, dxo, dh, post, gate, pre, given_ws});
        const OnStream on(a, 10, x);
        const Tensor none;
        const Tensor dx = output(none, "dx", x, {m.T, m.D}, m.type);
        const Tensor dy = y.defined() ? output(none, "dy", x, {m.T, m.D}, m.type) : none;
        const Tensor dpost = post.defined() ? output(none, "dgamma_post", x, {m.D}, m.ptype) : none;
        const Tensor dgate = gate.defined() ? output(none, "dgate", x, {m.G, m.D}, m.ptype) : none;
        const Tensor dpre = pre.defined() ? output(none, "dgamma_pre", x, {m.D}, m.ptype) : none;
        const Tensor ws = workspace(given_ws, given_ws.defined() ? 0 : moe_block_norm_backward_workspace_size(T, D, G), x);
        check(moe_block_norm_backward(m.dt, m.pt, T, D, G, a.number(7, 1.0), a.number(8, 1e-6), ptr(post), ptr(gate),
                                      ptr(pre), ptr(x), ptr(y), ptr(dxo), ptr(dh), ptr(dx), ptr(dy), ptr(dpost), ptr(dgate),
                                      ptr(dpre), ptr(ws), (size_t)ws.numel(), on.s), "moe_block_norm_backward");
        return wrap_all({dx, dy, dpost, dgate, dpre});
    });
}

PyObject* py_init(PyObject*, PyObject* check_fn) {
    Py_INCREF(check_fn);
    Py_XDECREF(g_check);
    g_check = check_fn;
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS
PyMethodDef methods[] = {
    {"grouped_mm", FAST(py_grouped_mm),
     "grouped_mm(x, w, offsets, y=None, ws=None, stream=None) -> y\n\n"
     "y[r] = w[e] x[r] for the rows r of every expert e: x [R, K], w [E, N, K], offsets [E + 1] of permute().\n"
     "Offsets out of order or range set the error word of ws, for get_device_error(ws); without ws it is lost."},
    {"grouped_mm_dx", FAST(py_grouped_mm_dx),
     "grouped_mm_dx(dy, w, offsets, dx=None, ws=None, stream=None) -> dx\n\n"
     "Gradient of grouped_mm in x: dx[r] = dy[r] w[e]."},
    {"grouped_mm_dw", FAST(py_grouped_mm_dw),
     "grouped_mm_dw(dy, x, offsets, dw=None, ws=None, stream=None) -> dw\n\n"
     "Gradient of grouped_mm in w: dw[e] = sum of dy[r]^T x[r] over the expert's rows."},
    {"swiglu", FAST(py_swiglu),
     "swiglu(gu, row_w=None, row_map=None, h=None, stream=None) -> h\n\n"
     "h[r] = row_w[row_map[r]] SiLU(gate) up for gu [R, 2F], gate then up; row_map is `sorted` of permute()."},
    {"swiglu_backward", FAST(py_swiglu_backward),
     "swiglu_backward(dh, gu, row_w=None, row_map=None, dgu=None, drow_w=None, stream=None) -> (dgu, drow_w)\n\n"
     "Gradients of swiglu: dgu [R, 2F], drow_w [R] fp32 (None without row_w)."},
    {"block_norm", FAST(py_block_norm),
     "block_norm(x, y=None, gamma_post=None, gate=None, gamma_pre=None, alpha=1.0, eps=1e-6, x_out=None, h=None,\n"
     "           stream=None) -> (x_out, h)\n\n"
     "x_out = x + alpha gate norm(y) gamma_post and h = norm(x_out) gamma_pre; x_out is None without y, h is None\n"
     "without gamma_pre.  gamma_post None: y enters unnormalised; gate [G, D] None: 1; x_out may be x."},
    {"block_norm_backward", FAST(py_block_norm_backward),
     "block_norm_backward(x_out, y=None, dx_out=None, dh=None, gamma_post=None, gate=None, gamma_pre=None, alpha=1.0,\n"
     "                    eps=1e-6, ws=None, stream=None) -> (dx, dy, dgamma_post, dgate, dgamma_pre)\n\n"
     "Gradients of block_norm at the stored x_out (x, where there is no y); None for what was not there."},
    {"_init", py_init, METH_O, "Sets the function that raises for a status."},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_expert16", "16-bit expert operators of libmoe_w4.so", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__expert16(void) { return PyModule_Create(&module); }
