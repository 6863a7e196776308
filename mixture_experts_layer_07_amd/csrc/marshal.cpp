// Native half of binding.py: argument checks and calls of libmoe's entry
// points without ctypes.  A layer's small calls are bound by the host, and the
// checks and conversions in Python cost more there than the launch itself (a
// one-token rmsnorm with every output, back to back: 8.3 us a call in Python,
// of which the launch is 2.7).
//
// Each entry point is called through its own type in moe.h, so the conversions
// follow the header: a pointer parameter takes a tensor of the call's device or
// None, a number a Python number that fits it.  The library itself is opened by
// binding.py; this module gets the functions' addresses.
#include <Python.h>

#include <c10/core/GradMode.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <limits>
#include <string>
#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/moe.h"

namespace {

PyObject* g_resolve = nullptr;  // name -> address (int), from binding.py
PyObject* g_failed = nullptr;   // (name, status): raises MoeError
PyObject* g_refuse = nullptr;   // (tensor, name, dtype, shape): raises what check() found
PyObject* g_get_device = nullptr;
PyObject* g_set_device = nullptr;
PyObject* g_stream = nullptr;

// ------------------------------------------------------------------- call
// What a call says of a tensor that requires grad: nothing, or what to do instead.
const char* const kSilent = nullptr;
const char* const kBackwardCall = "detach it or call under torch.no_grad(), and use the backward call";  // it has one
const char* const kNoGradient = "detach it or call under torch.no_grad()";

struct Call {
    const char* name;
    long index;          // device
    const char* instead;
};

bool convert(PyObject* o, const Call& c, void** out)
{
    if (o == Py_None) {
        *out = nullptr;
        return true;
    }
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: a buffer is a tensor or None, not %R", c.name, o);
        return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    // A result that autograd takes for a constant must not lose the caller's gradient without a word.
    // (The gradients' calls may well take such tensors: a caller's own products under autograd.)
    if (c.instead && t.requires_grad() && c10::GradMode::is_enabled()) {
        const std::string text =
            std::string(c.name) + ": a tensor requires grad, but the call records no graph; " + c.instead;
        if (PyErr_WarnEx(PyExc_UserWarning, text.c_str(), 3)) return false;  // warnings may be errors
    }
    if (!t.is_cuda() || t.device().index() != c.index) {
        PyErr_Format(PyExc_ValueError, "%s: a tensor on %s, expected cuda:%ld", c.name, t.device().str().c_str(),
                     c.index);
        return false;
    }
    *out = t.data_ptr();
    return true;
}

template <class T>
bool convert(PyObject* o, const Call& c, T* out)
{
    if constexpr (std::is_pointer_v<T>) {
        void* p;
        if (!convert(o, c, &p)) return false;
        *out = static_cast<T>(p);
    } else if constexpr (std::is_floating_point_v<T>) {
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) return false;
        *out = static_cast<T>(v);
    } else {
        PyObject* n = PyNumber_Index(o);
        if (!n) return false;
        const long long v = PyLong_AsLongLong(n);
        Py_DECREF(n);
        if (v == -1 && PyErr_Occurred()) return false;
        const bool fits = std::is_signed_v<T> ? v >= (long long)std::numeric_limits<T>::min() &&
                                                    v <= (long long)std::numeric_limits<T>::max()
                                              : v >= 0 && (unsigned long long)v <= std::numeric_limits<T>::max();
        if (!fits) {
            PyErr_Format(PyExc_OverflowError, "%s: %lld does not fit its parameter", c.name, v);
            return false;
        }
        *out = static_cast<T>(v);
    }
    return true;
}

// The integer that a torch function of (args) returns; -1 with an error set.
long long ask(PyObject* f, PyObject* arg)
{
    PyObject* r = arg ? PyObject_CallOneArg(f, arg) : PyObject_CallNoArgs(f);
    if (!r) return -1;
    const long long v = r == Py_None ? 0 : PyLong_AsLongLong(r);
    Py_DECREF(r);
    return v;
}

bool set_device(long index)
{
    PyObject* i = PyLong_FromLong(index);
    if (!i) return false;
    ask(g_set_device, i);
    Py_DECREF(i);
    return !PyErr_Occurred();
}

// Converts all parameters but the last, makes the device current, appends its
// current stream and calls.  -1 with a Python error set, else the status.
template <class... A, size_t... I>
int run(moe_status (*f)(A...), Call c, PyObject* const* args, Py_ssize_t n, std::index_sequence<I...>)
{
    std::tuple<A...> v{};
    constexpr Py_ssize_t want = sizeof...(A) - 1;
    static_assert(std::is_same_v<std::tuple_element_t<want, std::tuple<A...>>, void*>, "the last is the stream");
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments and the stream (got %zd)", c.name, want, n);
        return -1;
    }
    if (c.index < 0 && (c.index = (long)ask(g_get_device, nullptr)) < 0) return -1;
    if (!((I == (size_t)want || convert(args[I == (size_t)want ? 0 : I], c, &std::get<I>(v))) && ...)) return -1;
    const long before = (long)ask(g_get_device, nullptr);
    if (before < 0) return -1;
    PyObject* i = PyLong_FromLong(c.index);
    if (!i) return -1;
    const long long stream = ask(g_stream, i);
    Py_DECREF(i);
    if (stream == -1 && PyErr_Occurred()) return -1;
    std::get<want>(v) = reinterpret_cast<void*>(stream);
    if (before != c.index && !set_device(c.index)) return -1;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = std::apply(f, v);
    Py_END_ALLOW_THREADS
    if (before != c.index && !set_device(before)) return -1;
    return st;
}

template <class... A>
int run_any(moe_status (*f)(A...), const Call& c, PyObject* const* args, Py_ssize_t n)
{
    return run(f, c, args, n, std::index_sequence_for<A...>{});
}

struct Entry {
    const char* name;
    int (*run)(void*, const Call&, PyObject* const*, Py_ssize_t);
    const char* instead;
    void* address;
};

#define MOE_ENTRY(fn, instead)                                                                           \
    {                                                                                                    \
        #fn,                                                                                             \
            [](void* f, const Call& c, PyObject* const* a, Py_ssize_t n) {                               \
                return run_any(reinterpret_cast<decltype(&fn)>(f), c, a, n);                             \
            },                                                                                           \
            instead, nullptr                                                                             \
    }

Entry g_entries[] = {
    MOE_ENTRY(moe_route, kSilent),
    MOE_ENTRY(moe_permute, kSilent),
    MOE_ENTRY(moe_expert_ffn, kSilent),
    MOE_ENTRY(moe_expert_ffn_noalloc, kSilent),
    MOE_ENTRY(moe_expert_ffn_fp8, kSilent),
    MOE_ENTRY(moe_expert_ffn_fused, kSilent),
    MOE_ENTRY(moe_expert_ffn_fp8_fused, kSilent),
    MOE_ENTRY(moe_finalize, kSilent),
    MOE_ENTRY(moe_quantize_fp8, kSilent),
    MOE_ENTRY(moe_rmsnorm, kBackwardCall),
    MOE_ENTRY(moe_rmsnorm_backward, kSilent),
    MOE_ENTRY(moe_dispatch, kBackwardCall),
    MOE_ENTRY(moe_dispatch_backward, kSilent),
    MOE_ENTRY(moe_finalize_backward, kSilent),
    MOE_ENTRY(moe_route_backward, kSilent),
    MOE_ENTRY(moe_swiglu, kBackwardCall),
    MOE_ENTRY(moe_swiglu_backward, kSilent),
    MOE_ENTRY(moe_quantize_mxfp4, kNoGradient),
    MOE_ENTRY(moe_dequantize_mxfp4, kNoGradient),
    MOE_ENTRY(moe_expert_ffn_mxfp4, kNoGradient),
    MOE_ENTRY(moe_layer_few, kNoGradient),
};

// A tensor without storage of its own makes torch throw: no exception leaves
// this module.
template <class F>
PyObject* guarded(F f)
{
    try {
        return f();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// call(name, device, *arguments): MoeError for a status that is not MOE_OK.
PyObject* call_(PyObject* const* args, Py_ssize_t n)
{
    if (n < 2 || !PyUnicode_Check(args[0]) || !THPDevice_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "call(name, device, *arguments)");
        return nullptr;
    }
    const char* name = PyUnicode_AsUTF8(args[0]);
    if (!name) return nullptr;
    Entry* entry = nullptr;
    for (Entry& e : g_entries)
        if (!strcmp(e.name, name)) entry = &e;
    if (!entry) {
        PyErr_Format(PyExc_AttributeError, "no entry point %s", name);
        return nullptr;
    }
    const at::Device& dev = reinterpret_cast<THPDevice*>(args[1])->device;
    if (!entry->address) {
        const long long a = ask(g_resolve, args[0]);
        if (PyErr_Occurred()) return nullptr;
        entry->address = reinterpret_cast<void*>(a);
    }
    const int st = entry->run(entry->address, Call{entry->name, dev.has_index() ? (long)dev.index() : -1, entry->instead},
                              args + 2, n - 2);
    if (st < 0) return nullptr;
    if (st != MOE_OK) {
        PyObject* r = PyObject_CallFunction(g_failed, "si", name, st);
        Py_XDECREF(r);
        if (!r) return nullptr;
    }
    Py_RETURN_NONE;
}

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&] { return call_(args, n); });
}

// ------------------------------------------------------------------ check
bool has_type(const at::Tensor& t, PyObject* dtype)
{
    if (dtype == Py_None) return true;
    if (THPDtype_Check(dtype)) return t.scalar_type() == reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    if (!PyTuple_Check(dtype)) return false;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(dtype); ++i) {
        PyObject* d = PyTuple_GET_ITEM(dtype, i);
        if (THPDtype_Check(d) && t.scalar_type() == reinterpret_cast<THPDtype*>(d)->scalar_type) return true;
    }
    return false;
}

bool has_shape(const at::Tensor& t, PyObject* shape)
{
    if (shape == Py_None) return true;
    if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t.dim()) return false;
    for (Py_ssize_t i = 0; i < t.dim(); ++i) {
        const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();  // the Python form says what is wrong
            return false;
        }
        if (v != t.size(i)) return false;
    }
    return true;
}

// check(tensor, name, dtype=None, shape=None) -> tensor: a contiguous GPU
// tensor of that type (or one of a tuple of types) and shape, or ValueError.
PyObject* check_(PyObject* const* args, Py_ssize_t n, PyObject* kwnames)
{
    PyObject* a[4] = {nullptr, nullptr, Py_None, Py_None};
    if (n > 4) n = 5;
    for (Py_ssize_t i = 0; i < n && i < 4; ++i) a[i] = args[i];
    const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    bool bad = n > 4;
    for (Py_ssize_t i = 0; i < nk && !bad; ++i) {
        PyObject* k = PyTuple_GET_ITEM(kwnames, i);
        if (!PyUnicode_CompareWithASCIIString(k, "dtype")) a[2] = args[n + i];
        else if (!PyUnicode_CompareWithASCIIString(k, "shape")) a[3] = args[n + i];
        else bad = true;
    }
    if (bad || !a[0] || !a[1]) {
        PyErr_SetString(PyExc_TypeError, "check(tensor, name, dtype=None, shape=None)");
        return nullptr;
    }
    if (THPVariable_Check(a[0])) {
        const at::Tensor& t = THPVariable_Unpack(a[0]);
        if (t.is_cuda() && has_type(t, a[2]) && has_shape(t, a[3]) && t.is_contiguous()) {
            Py_INCREF(a[0]);
            return a[0];
        }
    }
    return PyObject_CallFunctionObjArgs(g_refuse, a[0], a[1], a[2], a[3], nullptr);
}

PyObject* check(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames)
{
    return guarded([&] { return check_(args, n, kwnames); });
}

// setup(resolve, failed, refuse)
PyObject* setup(PyObject*, PyObject* args)
{
    PyObject *r, *f, *u;
    if (!PyArg_ParseTuple(args, "OOO", &r, &f, &u)) return nullptr;
    PyObject* c = PyImport_ImportModule("torch._C");
    if (!c) return nullptr;
    PyObject* get = PyObject_GetAttrString(c, "_cuda_getDevice");
    PyObject* set = get ? PyObject_GetAttrString(c, "_cuda_setDevice") : nullptr;
    PyObject* stream = set ? PyObject_GetAttrString(c, "_cuda_getCurrentRawStream") : nullptr;
    Py_DECREF(c);
    if (!stream) {
        Py_XDECREF(get);
        Py_XDECREF(set);
        return nullptr;
    }
    Py_INCREF(r);
    Py_INCREF(f);
    Py_INCREF(u);
    std::swap(g_resolve, r);
    std::swap(g_failed, f);
    std::swap(g_refuse, u);
    std::swap(g_get_device, get);
    std::swap(g_set_device, set);
    std::swap(g_stream, stream);
    for (PyObject* o : {r, f, u, get, set, stream}) Py_XDECREF(o);
    for (Entry& e : g_entries) e.address = nullptr;
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(call)), METH_FASTCALL, nullptr},
    {"check", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(check)), METH_FASTCALL | METH_KEYWORDS, nullptr},
    {"setup", setup, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
