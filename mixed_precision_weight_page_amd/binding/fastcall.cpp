// The ordinary call of the package's context-free operators, from Python
// straight to the C ABI: tensors are looked at through torch's C++ interface,
// new outputs come from its allocator, and the library's function runs on the
// current stream. Every function returns None for anything that is not such a
// call (a wrong type, shape, device or distance, a gradient or tangent that would
// be lost, a status that is not 0), and the Python function of the same name then
// goes through its own checks, which say what is wrong. (Host time of a call
// of linear_fp8 through ctypes 9.6 us, so 5; the smallest kernels take 3.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pagedweight.h"

namespace {

using at::Tensor;

// the library's functions, once it is loaded
struct Library {
    decltype(&pw_rms_norm) rms_norm;
    decltype(&pw_quantize_fp8) quantize_fp8;
    decltype(&pw_linear_fp8) linear_fp8;
    decltype(&pw_grouped_linear) grouped_linear;
} lib{};

constexpr int kNone = -1;
int code_of(c10::ScalarType t) {
    switch (t) {
        case c10::ScalarType::Float: return PW_F32;
        case c10::ScalarType::Half: return PW_F16;
        case c10::ScalarType::BFloat16: return PW_BF16;
        case c10::ScalarType::Float8_e4m3fn: return PW_E4M3;
        default: return kNone;
    }
}
bool wide(int code) { return code == PW_F32 || code == PW_F16 || code == PW_BF16; }
int64_t blocks(int64_t n) { return (n + 127) / 128; }

// A call's view of its arguments: `ok` turns false at the first that is not
// what an ordinary call has.
struct Call {
    bool ok = true;
    c10::DeviceIndex dev = -1;

    // a tensor on the call's device; the first one sets it
    const Tensor* tensor(PyObject* o) {
        if (!ok || !THPVariable_Check(o)) return no();
        const Tensor& t = THPVariable_Unpack(o);
        if (!t.defined() || !t.is_cuda() || t.unsafeGetTensorImpl()->is_python_dispatch() ||
            t.layout() != c10::kStrided || (t.requires_grad() && c10::GradMode::is_enabled()) ||
            t._fw_grad(0).defined())   // a forward-mode tangent
            return no();
        if (dev < 0) {
            dev = t.device().index();
            if (dev != c10::hip::current_device()) return no();
        } else if (t.device().index() != dev) {
            return no();
        }
        return &t;
    }
    const Tensor* maybe(PyObject* o) { return o == Py_None ? nullptr : tensor(o); }
    void need(bool condition) { ok = ok && condition; }

    // contiguous rows, any other distances
    void rows(const Tensor* t, int64_t n, int64_t cols) {
        if (!ok) return;
        need(t->dim() == 2 && t->size(0) == n && t->size(1) == cols && (cols <= 1 || t->stride(1) == 1));
    }
    void vector(const Tensor* t, c10::ScalarType type, int64_t n) {
        if (!ok || !t) return;
        need(t->scalar_type() == type && t->dim() == 1 && t->size(0) == n && t->is_contiguous());
    }
    void scales(const Tensor* t, int64_t n, int64_t cols) {
        if (!ok) return;
        need(t->scalar_type() == c10::ScalarType::Float && t->dim() == 2 && t->size(0) == n && t->size(1) == cols);
    }
    // codes and scales
    bool pair(PyObject* o, const Tensor** q, const Tensor** s) {
        need(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2);
        if (!ok) return false;
        *q = tensor(PyTuple_GET_ITEM(o, 0));
        *s = tensor(PyTuple_GET_ITEM(o, 1));
        return ok;
    }
    void* stream() const { return c10::hip::getCurrentHIPStream(dev).stream(); }

private:
    const Tensor* no() {
        ok = false;
        return nullptr;
    }
};

c10::TensorOptions like(const Tensor& t, c10::ScalarType type) { return t.options().dtype(type).requires_grad(false); }
void* at_of(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
float* floats(const Tensor* t) { return static_cast<float*>(at_of(t)); }

// out_dtype, else the type of the first of these that is given, else `type`
bool out_type(Call& c, PyObject* o, const Tensor* y, const Tensor* residual, c10::ScalarType* type) {
    if (o != Py_None) {
        c.need(THPDtype_Check(o));
        if (c.ok) *type = reinterpret_cast<THPDtype*>(o)->scalar_type;
    } else if (y || residual) {
        *type = (y ? y : residual)->scalar_type();
    }
    c.need(c.ok && wide(code_of(*type)));
    return c.ok;
}

PyObject* none() { Py_RETURN_NONE; }

// (x, weight, eps, residual, h, out_dtype): y or (codes, scales), with a
// residual (that, h); a given `out` is no ordinary call
PyObject* rms_norm(PyObject* const* args, Py_ssize_t n_args) {
    if (n_args != 6 || !lib.rms_norm) return none();
    Call c;
    const Tensor* x = c.tensor(args[0]);
    if (!c.ok || x->dim() != 2) return none();
    const int64_t T = x->size(0), n = x->size(1);
    c.rows(x, T, n);
    const Tensor* weight = c.maybe(args[1]);
    const double eps = PyFloat_Check(args[2]) ? PyFloat_AS_DOUBLE(args[2]) : -1.0;
    const Tensor* residual = c.maybe(args[3]);
    const Tensor* given = c.maybe(args[4]);
    c10::ScalarType type = x->scalar_type();
    if (args[5] != Py_None) {
        c.need(THPDtype_Check(args[5]));
        if (c.ok) type = reinterpret_cast<THPDtype*>(args[5])->scalar_type;
    }
    const int out = code_of(type), xt = code_of(x->scalar_type());
    c.need(out != kNone && wide(xt) && eps >= 0.0 && (residual || !given) && T <= INT32_MAX && n <= INT32_MAX);
    if (c.ok && weight) {
        c.need(wide(code_of(weight->scalar_type())));
        c.vector(weight, weight->scalar_type(), n);
    }
    if (c.ok && residual) {
        c.need(residual->scalar_type() == x->scalar_type() || residual->scalar_type() == c10::ScalarType::Float);
        c.rows(residual, T, n);
        if (c.ok && given) {
            c.need(given->scalar_type() == residual->scalar_type());
            c.rows(given, T, n);
        }
    }
    if (!c.ok) return none();
    const bool eight = out == PW_E4M3;
    const int64_t ld = eight ? (n + 15) & ~(int64_t)15 : n;
    Tensor y = eight ? at::empty_strided({T, n}, {ld, 1}, like(*x, type)) : at::empty({T, n}, like(*x, type));
    Tensor scale, h;
    if (eight) scale = at::empty_strided({T, blocks(n)}, {1, T}, like(*x, c10::ScalarType::Float));
    if (residual) h = given ? *given : at::empty({T, n}, like(*x, residual->scalar_type()));
    const pw_rms_norm_desc d = {(int32_t)T, (int32_t)n, xt, residual ? code_of(residual->scalar_type()) : 0,
                                weight ? code_of(weight->scalar_type()) : 0, out, x->stride(0),
                                residual ? residual->stride(0) : n, residual ? h.stride(0) : n, ld, 1, T, (float)eps};
    if (lib.rms_norm(&d, x->data_ptr(), at_of(weight), at_of(residual), residual ? h.data_ptr() : nullptr, y.data_ptr(),
                     eight ? static_cast<float*>(scale.data_ptr()) : nullptr, c.stream()) != PW_OK)
        return none();
    return eight ? (residual ? Py_BuildValue("NNN", THPVariable_Wrap(y), THPVariable_Wrap(scale), THPVariable_Wrap(h))
                             : Py_BuildValue("NN", THPVariable_Wrap(y), THPVariable_Wrap(scale)))
                 : (residual ? Py_BuildValue("NN", THPVariable_Wrap(y), THPVariable_Wrap(h)) : THPVariable_Wrap(y));
}

// (x, tile): (codes, scales)
PyObject* quantize_fp8(PyObject* const* args, Py_ssize_t n_args) {
    if (n_args != 2 || !lib.quantize_fp8) return none();
    Call c;
    const Tensor* x = c.tensor(args[0]);
    const bool tile = args[1] == Py_True;
    if (!c.ok || (x->dim() != 2 && x->dim() != 3)) return none();
    const bool batched = x->dim() == 3;
    const int64_t E = batched ? x->size(0) : 1, M = x->size(-2), K = x->size(-1);
    c.need(wide(code_of(x->scalar_type())) && (K <= 1 || x->stride(-1) == 1) && E <= INT32_MAX && M <= INT32_MAX && K <= INT32_MAX);
    if (!c.ok) return none();
    const int64_t ld = (K + 15) & ~(int64_t)15, down = tile ? blocks(M) : M, KB = blocks(K);
    Tensor q, scale;
    const auto codes = like(*x, c10::ScalarType::Float8_e4m3fn), fp32 = like(*x, c10::ScalarType::Float);
    const int64_t s_row = tile ? KB : 1, s_block = tile ? 1 : M, s_batch = down * KB;
    if (batched) {
        q = at::empty_strided({E, M, K}, {M * ld, ld, 1}, codes);
        scale = at::empty_strided({E, down, KB}, {s_batch, s_row, s_block}, fp32);
    } else {
        q = at::empty_strided({M, K}, {ld, 1}, codes);
        scale = at::empty_strided({down, KB}, {s_row, s_block}, fp32);
    }
    const pw_quantize_desc d = {(int32_t)E, (int32_t)M, (int32_t)K, code_of(x->scalar_type()), tile, x->stride(-2),
                                batched ? x->stride(0) : 0, ld, batched ? M * ld : 0, s_row, s_block, batched ? s_batch : 0};
    if (lib.quantize_fp8(&d, x->data_ptr(), q.data_ptr(), static_cast<float*>(scale.data_ptr()), c.stream()) != PW_OK) return none();
    return Py_BuildValue("NN", THPVariable_Wrap(q), THPVariable_Wrap(scale));
}

// (x, w, bias, act, residual, y, out_dtype): y
PyObject* linear_fp8(PyObject* const* args, Py_ssize_t n_args) {
    if (n_args != 7 || !lib.linear_fp8 || !PyLong_Check(args[3])) return none();
    Call c;
    const Tensor *x, *xs, *w, *ws;
    if (!c.pair(args[0], &x, &xs) || !c.pair(args[1], &w, &ws)) return none();
    const int act = (int)PyLong_AsLong(args[3]), halves = act == PW_ACT_SWIGLU ? 2 : 1;
    if (x->dim() != 2 || w->dim() != 2 || w->size(0) % halves) return none();
    const int64_t M = x->size(0), K = x->size(1), R = w->size(0), N = R / halves;
    c.need(code_of(x->scalar_type()) == PW_E4M3 && code_of(w->scalar_type()) == PW_E4M3 && M <= INT32_MAX && R <= INT32_MAX &&
           K <= INT32_MAX);
    c.rows(x, M, K);
    c.rows(w, R, K);
    c.scales(xs, M, blocks(K));
    c.scales(ws, halves * blocks(N), blocks(K));
    const Tensor *bias = c.maybe(args[2]), *residual = c.maybe(args[4]), *given = c.maybe(args[5]);
    c.vector(bias, c10::ScalarType::Float, R);
    c10::ScalarType type = c10::ScalarType::BFloat16;
    if (!c.ok || !out_type(c, args[6], given, residual, &type)) return none();
    for (const Tensor* t : {residual, given}) {
        if (!t) continue;
        c.need(t->scalar_type() == type);
        c.rows(t, M, N);
    }
    if (!c.ok) return none();
    const Tensor y = given ? *given : at::empty({M, N}, like(*x, type));
    const pw_linear_fp8_desc d = {(int32_t)M, (int32_t)N, (int32_t)K, code_of(type), act, x->stride(0), w->stride(0),
                                  residual ? residual->stride(0) : N, y.stride(0), xs->stride(0), xs->stride(1), ws->stride(0),
                                  ws->stride(1)};
    if (lib.linear_fp8(&d, x->data_ptr(), floats(xs), w->data_ptr(), floats(ws), floats(bias), at_of(residual), y.data_ptr(),
                       c.stream()) != PW_OK)
        return none();
    return THPVariable_Wrap(y);
}

// (x, offsets, w, bias, act, residual, y, rows, out_dtype): y
PyObject* grouped_linear(PyObject* const* args, Py_ssize_t n_args) {
    if (n_args != 9 || !lib.grouped_linear || !PyLong_Check(args[4])) return none();
    Call c;
    const Tensor *x, *xs = nullptr, *w, *ws = nullptr;
    const bool eight = PyTuple_Check(args[0]);
    if (eight) {
        if (!c.pair(args[0], &x, &xs) || !c.pair(args[2], &w, &ws)) return none();
    } else {
        x = c.tensor(args[0]);
        w = c.tensor(args[2]);
    }
    const Tensor* offsets = c.tensor(args[1]);
    const int act = (int)PyLong_AsLong(args[4]), halves = act == PW_ACT_SWIGLU ? 2 : 1;
    if (!c.ok || x->dim() != 2 || w->dim() != 3 || w->size(1) % halves) return none();
    const int64_t x_rows = x->size(0), K = x->size(1), E = w->size(0), R = w->size(1), N = R / halves;
    const int in = code_of(x->scalar_type());
    const Tensor *bias = c.maybe(args[3]), *residual = c.maybe(args[5]), *given = c.maybe(args[6]), *rows = c.maybe(args[7]);
    if (!c.ok || (rows && rows->dim() != 1)) return none();
    const int64_t M = rows ? rows->size(0) : x_rows;
    c.need((eight ? in == PW_E4M3 : in == PW_F16 || in == PW_BF16) && w->scalar_type() == x->scalar_type() && w->size(2) == K &&
           (K <= 1 || w->stride(2) == 1) && M <= INT32_MAX && x_rows <= INT32_MAX && R <= INT32_MAX && K <= INT32_MAX &&
           E <= INT32_MAX);
    c.rows(x, x_rows, K);
    if (eight) {
        c.scales(xs, x_rows, blocks(K));
        c.need(ws->scalar_type() == c10::ScalarType::Float && ws->dim() == 3 && ws->size(0) == E &&
               ws->size(1) == halves * blocks(N) && ws->size(2) == blocks(K));
    }
    c.vector(offsets, c10::ScalarType::Int, E + 1);
    c.vector(rows, c10::ScalarType::Int, M);
    if (c.ok && bias)
        c.need(bias->scalar_type() == c10::ScalarType::Float && bias->dim() == 2 && bias->size(0) == E && bias->size(1) == R &&
               bias->is_contiguous());
    c10::ScalarType type = eight ? c10::ScalarType::BFloat16 : x->scalar_type();
    if (!c.ok || !out_type(c, args[8], given, residual, &type)) return none();
    for (const Tensor* t : {residual, given}) {
        if (!t) continue;
        c.need(t->scalar_type() == type);
        c.rows(t, M, N);
    }
    if (!c.ok) return none();
    const Tensor y = given ? *given : at::empty({M, N}, like(*x, type));
    const pw_grouped_desc d = {(int32_t)M, (int32_t)N, (int32_t)K, (int32_t)E, (int32_t)x_rows, in, code_of(type), act,
                               x->stride(0), w->stride(1), w->stride(0), residual ? residual->stride(0) : N, y.stride(0),
                               eight ? xs->stride(0) : 0, eight ? xs->stride(1) : 0, eight ? ws->stride(1) : 0,
                               eight ? ws->stride(2) : 0, eight ? ws->stride(0) : 0};
    if (lib.grouped_linear(&d, x->data_ptr(), floats(xs), w->data_ptr(), floats(ws),
                           static_cast<const int32_t*>(offsets->data_ptr()), static_cast<const int32_t*>(at_of(rows)),
                           floats(bias), at_of(residual), y.data_ptr(), c.stream()) != PW_OK)
        return none();
    return THPVariable_Wrap(y);
}

// What torch throws (no memory, for one) is left to the Python function's own
// attempt, which raises it.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        return F(args, n);
    } catch (...) {
        PyErr_Clear();
        return none();
    }
}

// (addresses of pw_rms_norm, pw_quantize_fp8, pw_linear_fp8, pw_grouped_linear)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "four addresses");
        return nullptr;
    }
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (!p[i] && PyErr_Occurred()) return nullptr;
    }
    lib.rms_norm = reinterpret_cast<decltype(lib.rms_norm)>(p[0]);
    lib.quantize_fp8 = reinterpret_cast<decltype(lib.quantize_fp8)>(p[1]);
    lib.linear_fp8 = reinterpret_cast<decltype(lib.linear_fp8)>(p[2]);
    lib.grouped_linear = reinterpret_cast<decltype(lib.grouped_linear)>(p[3]);
    Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F* f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"rms_norm", fast(guarded<rms_norm>), METH_FASTCALL, nullptr},
                         {"quantize_fp8", fast(guarded<quantize_fp8>), METH_FASTCALL, nullptr},
                         {"linear_fp8", fast(guarded<linear_fp8>), METH_FASTCALL, nullptr},
                         {"grouped_linear", fast(guarded<grouped_linear>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
