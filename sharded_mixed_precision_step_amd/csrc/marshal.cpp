// The binding's short ways, since a short call's time is the host's (a layer norm of 16
// rows: 9.5 us a call with lookups in Python and ctypes, 4.6 of them the kernel's).
//
// mat, like, vec, q8: what train.py reads off a tensor for a call: device pointer, type
// code, row stride.  Each has the signature of the Python function it stands for and
// answers where everything is as it should be; anything else goes to that Python
// function, which init() is given, and which raises what there is to raise.
//
// zero_*: the calls of zero_model.h on numbers, as ctypes makes them, by the addresses
// that bind() is given: None is NULL, the result is the status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits>
#include <type_traits>

#include <torch/csrc/Device.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "zero_model.h"

namespace {

PyObject* g_checked[4];  // mat, like, vec, q8 in Python

PyObject* checked(int which, PyObject* const* args, Py_ssize_t n) {
    if (!g_checked[which]) {
        PyErr_SetString(PyExc_RuntimeError, "marshal: init() has not been called");
        return nullptr;
    }
    return PyObject_Vectorcall(g_checked[which], args, static_cast<size_t>(n), nullptr);
}

// The tensor behind obj if it is on device dev and its type is among kinds; its code.
const at::Tensor* tensor(PyObject* obj, PyObject* kinds, PyObject* dev, long* code) {
    if (!THPVariable_Check(obj) || !PyDict_CheckExact(kinds) || !THPDevice_Check(dev))
        return nullptr;
    const at::Tensor& t = THPVariable_Unpack(obj);
    if (t.layout() != at::kStrided || t.device() != reinterpret_cast<THPDevice*>(dev)->device)
        return nullptr;
    PyObject* dtype = reinterpret_cast<PyObject*>(torch::getTHPDtype(t.scalar_type()));
    PyObject* found = PyDict_GetItemWithError(kinds, dtype);
    if (!found) {
        PyErr_Clear();
        return nullptr;
    }
    *code = PyLong_AsLong(found);
    return &t;
}

// The row stride of a matrix with contiguous rows.  A single row's says nothing: it
// counts as the row's length, rounded up to what the q8 layout asks of strides.
bool row_stride(const at::Tensor& t, int64_t* ld) {
    if (t.dim() != 2) return false;
    const int64_t rows = t.size(0), cols = t.size(1);
    if (cols > 1 && t.stride(1) != 1) return false;
    *ld = rows <= 1 ? (cols + 15) & -16 : t.stride(0);
    return true;
}

PyObject* pointer(const at::Tensor& t) {
    return PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t.data_ptr()));
}

// Steals the references; NULL if one is.
PyObject* tuple(std::initializer_list<PyObject*> items) {
    PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    Py_ssize_t k = 0;
    bool whole = out != nullptr;
    for (PyObject* item : items) {
        if (!item) whole = false;
        if (out) PyTuple_SET_ITEM(out, k++, item);
        else Py_XDECREF(item);
    }
    if (!whole) Py_CLEAR(out);
    return out;
}

PyObject* three(const at::Tensor& t, long code, int64_t ld) {
    return tuple({pointer(t), PyLong_FromLong(code), PyLong_FromLongLong(ld)});
}

// A C++ exception of torch's ends at the C boundary as a Python one.
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// mat(tensor, kinds, dev, name)
PyObject* mat(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        long code = 0;
        int64_t ld = 0;
        const at::Tensor* t = n == 4 ? tensor(a[0], a[1], a[2], &code) : nullptr;
        if (!t || !row_stride(*t, &ld)) return checked(0, a, n);
        return three(*t, code, ld);
    });
}

// like(tensor, shape, kinds, dev, name)
PyObject* like(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        long code = 0;
        int64_t ld = 0;
        const at::Tensor* t = n == 5 ? tensor(a[0], a[2], a[3], &code) : nullptr;
        if (!t || !row_stride(*t, &ld) || !PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 2)
            return checked(1, a, n);
        for (int k = 0; k < 2; ++k) {
            PyObject* want = PyTuple_GET_ITEM(a[1], k);
            if (!PyLong_Check(want) || PyLong_AsLongLong(want) != t->size(k)) {
                PyErr_Clear();
                return checked(1, a, n);
            }
        }
        return three(*t, code, ld);
    });
}

// vec(tensor, n, kinds, dev, name)
PyObject* vec(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        long code = 0;
        const at::Tensor* t = n == 5 ? tensor(a[0], a[2], a[3], &code) : nullptr;
        if (!t || !PyLong_Check(a[1]) || PyLong_AsLongLong(a[1]) != t->numel() ||
            !t->is_contiguous()) {
            PyErr_Clear();
            return checked(2, a, n);
        }
        return tuple({pointer(*t), PyLong_FromLong(code)});
    });
}

PyObject *g_fp8, *g_scale;  // the kinds of q8 data and scales

// q8(data, scales, rows, cols, dev, name, fmt=None)
PyObject* q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n < 6 || n > 7 || !g_fp8) return checked(3, a, n);
        PyObject* fmt = n == 7 ? a[6] : Py_None;
        if (a[0] == Py_None && a[1] == Py_None) {
            Py_INCREF(Py_None);
            Py_INCREF(Py_None);
            Py_INCREF(fmt);
            return tuple({Py_None, PyLong_FromLong(0), Py_None, PyLong_FromLong(0), fmt});
        }
        long code = 0, unused = 0;
        int64_t ld = 0, ld_s = 0;
        const at::Tensor* t = tensor(a[0], g_fp8, a[4], &code);
        const at::Tensor* s = tensor(a[1], g_scale, a[4], &unused);
        if (!t || !s || !row_stride(*t, &ld) || !row_stride(*s, &ld_s) || !PyLong_Check(a[2]) ||
            !PyLong_Check(a[3]))
            return checked(3, a, n);
        const int64_t rows = PyLong_AsLongLong(a[2]), cols = PyLong_AsLongLong(a[3]);
        const int64_t blocks = (cols + 127) / 128;
        if (PyErr_Occurred() || cols < 0 || cols > (int64_t{1} << 60) || t->size(0) != rows ||
            s->size(0) != rows || t->size(1) < blocks * 128 || s->size(1) < (blocks + 3) / 4 * 4 ||
            (fmt != Py_None && (!PyLong_Check(fmt) || PyLong_AsLong(fmt) != code))) {
            PyErr_Clear();
            return checked(3, a, n);
        }
        return tuple({pointer(*t), PyLong_FromLongLong(ld), pointer(*s), PyLong_FromLongLong(ld_s),
                      PyLong_FromLong(code)});
    });
}

// init(mat, like, vec, q8, fp8, scale): the Python functions, and the kinds of q8's
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6 || !PyDict_CheckExact(a[4]) || !PyDict_CheckExact(a[5])) {
        PyErr_SetString(PyExc_TypeError, "init takes four functions and two dicts");
        return nullptr;
    }
    for (int k = 0; k < 4; ++k) {
        Py_INCREF(a[k]);
        Py_XSETREF(g_checked[k], a[k]);
    }
    Py_INCREF(a[4]);
    Py_XSETREF(g_fp8, a[4]);
    Py_INCREF(a[5]);
    Py_XSETREF(g_scale, a[5]);
    Py_RETURN_NONE;
}

#define ZERO_CALLS(X)                                                                   \
    X(zero_embed) X(zero_embed_backward) X(zero_layernorm) X(zero_layernorm_backward)   \
    X(zero_act) X(zero_act_backward) X(zero_logprob) X(zero_logprob_backward)

#define ZERO_INDEX(name) k_##name,
enum { ZERO_CALLS(ZERO_INDEX) kCalls };
#undef ZERO_INDEX
#define ZERO_NAME(name) #name,
const char* const g_names[] = {ZERO_CALLS(ZERO_NAME)};
#undef ZERO_NAME
void* g_calls[kCalls];

// A Python number as a C argument; false with a Python error.
template <class T>
bool convert(PyObject* o, T* out) {
    if constexpr (std::is_pointer_v<T>) {
        *out = o == Py_None ? nullptr : static_cast<T>(PyLong_AsVoidPtr(o));
        return *out || o == Py_None || !PyErr_Occurred();
    } else if constexpr (std::is_floating_point_v<T>) {
        const double v = PyFloat_AsDouble(o);
        *out = static_cast<T>(v);
        return v != -1.0 || !PyErr_Occurred();
    } else {
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) return false;
        if (v < std::numeric_limits<T>::min() || v > std::numeric_limits<T>::max()) {
            PyErr_Format(PyExc_OverflowError, "%lld is out of range", v);
            return false;
        }
        *out = static_cast<T>(v);
        return true;
    }
}

template <int I, class F>
struct Call;
template <int I, class... A>
struct Call<I, int(A...)> {
    template <size_t... K>
    static PyObject* make(PyObject* const* a, std::index_sequence<K...>) {
        std::tuple<A...> v;
        if (!(convert(a[K], &std::get<K>(v)) && ...)) return nullptr;
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = reinterpret_cast<int (*)(A...)>(g_calls[I])(std::get<K>(v)...);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(rc);
    }
    static PyObject* run(PyObject*, PyObject* const* a, Py_ssize_t n) {
        if (!g_calls[I] || n != static_cast<Py_ssize_t>(sizeof...(A))) {
            PyErr_Format(PyExc_TypeError, "%s takes %d arguments, and bind() first", g_names[I],
                         static_cast<int>(sizeof...(A)));
            return nullptr;
        }
        return make(a, std::index_sequence_for<A...>{});
    }
};

// bind({name: address})
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 1 || !PyDict_CheckExact(a[0])) {
        PyErr_SetString(PyExc_TypeError, "bind takes a dict of addresses");
        return nullptr;
    }
    for (int k = 0; k < kCalls; ++k) {
        PyObject* at = PyDict_GetItemString(a[0], g_names[k]);
        if (!at || !(g_calls[k] = PyLong_AsVoidPtr(at))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, g_names[k]);
            return nullptr;
        }
    }
    Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

#define ZERO_METHOD(name) \
    {#name, fast(Call<k_##name, decltype(::name)>::run), METH_FASTCALL, nullptr},
PyMethodDef methods[] = {
    {"mat", fast(mat), METH_FASTCALL, nullptr},   {"like", fast(like), METH_FASTCALL, nullptr},
    {"vec", fast(vec), METH_FASTCALL, nullptr},   {"q8", fast(q8), METH_FASTCALL, nullptr},
    {"init", fast(init), METH_FASTCALL, nullptr}, {"bind", fast(bind), METH_FASTCALL, nullptr},
    ZERO_CALLS(ZERO_METHOD) {nullptr, nullptr, 0, nullptr}};
#undef ZERO_METHOD

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
