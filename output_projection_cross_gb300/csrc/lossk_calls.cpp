// lossk_calls.cpp -- the decoding calls as a CPython module: arguments by
// position, in the order of lossk.h, None for NULL, the status returned.  And
// spans() and device(), the checks and addresses of the tensors that such a call
// takes.
//
// A decoding step makes several of these calls per layer, of 13 to 30
// arguments each; through ctypes such a call took 2 us for its arguments
// alone, as long as its checks or its launch.  The functions are those of the
// library that load() names, so the module links nothing of it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/lossk.h"

#include <dlfcn.h>

#include <type_traits>
#include <tuple>
#include <utility>

namespace {

#define LOSSK_CALLS(X)                                                                                                \
    X(lossk_beam_select) X(lossk_beam_gather) X(lossk_cache_fork) X(lossk_cache_reserve) X(lossk_cache_free)          \
    X(lossk_cache_compact) X(lossk_cache_copy) X(lossk_cache_write) X(lossk_paged_attn)

enum Call {
#define X(name) CALL_##name,
    LOSSK_CALLS(X)
#undef X
    N_CALLS
};
void *address[N_CALLS];

// One argument; an error stays set in the interpreter.
template <typename A> A argument(PyObject *o)
{
    if constexpr (std::is_floating_point<A>::value) {
        return static_cast<A>(PyFloat_AsDouble(o));
    } else if constexpr (std::is_pointer<A>::value) {
        return o == Py_None ? nullptr : reinterpret_cast<A>(PyLong_AsUnsignedLongLong(o));
    } else {
        const long long x = PyLong_AsLongLong(o);
        if (static_cast<long long>(static_cast<A>(x)) != x) PyErr_SetString(PyExc_OverflowError, "argument out of range");
        return static_cast<A>(x);
    }
}

template <typename F> struct Caller;
template <typename R, typename... A> struct Caller<R(A...)> {
    template <size_t... I> static PyObject *run(R (*f)(A...), PyObject *const *a, std::index_sequence<I...>)
    {
        const std::tuple<A...> x{argument<A>(a[I])...};
        if (PyErr_Occurred()) return nullptr;
        R r;
        Py_BEGIN_ALLOW_THREADS
        r = f(std::get<I>(x)...);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(r);
    }
    static PyObject *call(void *f, PyObject *const *a, Py_ssize_t n)
    {
        if (n != sizeof...(A)) {
            PyErr_Format(PyExc_TypeError, "%zd arguments where %zu are needed", n, sizeof...(A));
            return nullptr;
        }
        if (!f) {
            PyErr_SetString(PyExc_RuntimeError, "the library has not been loaded");
            return nullptr;
        }
        return run(reinterpret_cast<R (*)(A...)>(f), a, std::index_sequence_for<A...>());
    }
};

#define X(name)                                                                                                       \
    PyObject *py_##name(PyObject *, PyObject *const *a, Py_ssize_t n)                                                 \
    {                                                                                                                 \
        return Caller<decltype(name)>::call(address[CALL_##name], a, n);                                              \
    }
LOSSK_CALLS(X)
#undef X

// Attributes and methods of a tensor.
PyObject *s_is_cuda, *s_dtype, *s_is_contiguous, *s_data_ptr, *s_numel, *s_get_device;

// Whether an attribute (or what a method returns) is the object `want`.
bool is(PyObject *got, PyObject *want)
{
    Py_XDECREF(got);
    return got == want;
}

// spans(dtype, t0, t1, ...): (address, elements) of each, flat, where all are
// contiguous CUDA tensors of that type; None, and no error, where one is not.  A
// t that is None counts as no elements at address 0.
PyObject *spans(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n < 1) {
        PyErr_SetString(PyExc_TypeError, "spans needs a type");
        return nullptr;
    }
    PyObject *r = PyTuple_New(2 * (n - 1));
    if (!r) return nullptr;
    for (Py_ssize_t i = 1; i < n; ++i) {
        PyObject *t = a[i], *p, *k;
        if (t == Py_None) {
            p = PyLong_FromLong(0);
            k = PyLong_FromLong(0);
        } else if (is(PyObject_GetAttr(t, s_is_cuda), Py_True) && is(PyObject_GetAttr(t, s_dtype), a[0]) &&
                   is(PyObject_CallMethodNoArgs(t, s_is_contiguous), Py_True)) {
            p = PyObject_CallMethodNoArgs(t, s_data_ptr);
            k = PyObject_CallMethodNoArgs(t, s_numel);
        } else {
            Py_DECREF(r);
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        if (p) PyTuple_SET_ITEM(r, 2 * (i - 1), p);
        if (k) PyTuple_SET_ITEM(r, 2 * (i - 1) + 1, k);
        if (!p || !k) {
            Py_DECREF(r);
            return nullptr;
        }
    }
    return r;
}

// device(t0, t1, ...): the index of the GPU that the tensors (None left out) are
// on; -1 where one is on none or on another than those before it.
PyObject *device(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    long all = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (a[i] == Py_None) continue;
        PyObject *got = PyObject_CallMethodNoArgs(a[i], s_get_device);
        if (!got) return nullptr;
        const long index = PyLong_AsLong(got);
        Py_DECREF(got);
        if (index == -1 && PyErr_Occurred()) return nullptr;
        if (index < 0 || (all >= 0 && index != all)) return PyLong_FromLong(-1);
        all = index;
    }
    return PyLong_FromLong(all);
}

// load(path): the library's functions.
PyObject *load(PyObject *, PyObject *path)
{
    const char *p = PyUnicode_AsUTF8(path);
    if (!p) return nullptr;
    void *lib = dlopen(p, RTLD_NOW);
    if (!lib) {
        PyErr_SetString(PyExc_OSError, dlerror());
        return nullptr;
    }
    const char *names[N_CALLS] = {
#define X(name) #name,
        LOSSK_CALLS(X)
#undef X
    };
    for (int i = 0; i < N_CALLS; ++i)
        if (!(address[i] = dlsym(lib, names[i]))) {
            PyErr_SetString(PyExc_OSError, dlerror());
            return nullptr;
        }
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"load", load, METH_O, nullptr},
    {"spans", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(spans)), METH_FASTCALL, nullptr},
    {"device", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(device)), METH_FASTCALL, nullptr},
#define X(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr},
    LOSSK_CALLS(X)
#undef X
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lossk_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__lossk_calls(void)
{
    const std::pair<PyObject **, const char *> names[] = {{&s_is_cuda, "is_cuda"},
                                                          {&s_dtype, "dtype"},
                                                          {&s_is_contiguous, "is_contiguous"},
                                                          {&s_data_ptr, "data_ptr"},
                                                          {&s_numel, "numel"},
                                                          {&s_get_device, "get_device"}};
    for (const auto &x : names)
        if (!(*x.first = PyUnicode_InternFromString(x.second))) return nullptr;
    return PyModule_Create(&module);
}
