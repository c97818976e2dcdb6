// py_calls.cpp -- the entry points of the cache and of the feed-forward layers as
// Python calls (module _calls).
//
// A decode step makes these calls for every layer, on kernels of a few
// microseconds, so the call itself counts.  With some twenty arguments ctypes
// took 3.0 us of a 5.3 us append (its conversions go by the argument, and each
// address is one more Python call); here the arguments come as an array and are
// converted by the types of the C prototype.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <climits>
#include <tuple>
#include <utility>

#include "bsk.h"

namespace {

PyObject* g_data_ptr;   // interned method and attribute names
PyObject* g_ctypes;
PyObject* g_data;

// A tensor's address, an address itself, None, or a NumPy array's.
bool address(PyObject* o, void** out)
{
    *out = nullptr;
    if (o == Py_None) return true;
    PyObject* r;
    if (PyLong_Check(o)) {
        r = Py_NewRef(o);
    } else {
        r = PyObject_CallMethodNoArgs(o, g_data_ptr);
        if (r == nullptr && PyErr_ExceptionMatches(PyExc_AttributeError)) {
            PyErr_Clear();
            PyObject* c = PyObject_GetAttr(o, g_ctypes);
            if (c == nullptr) return false;
            r = PyObject_GetAttr(c, g_data);
            Py_DECREF(c);
        }
        if (r == nullptr) return false;
    }
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return *out != nullptr || PyErr_Occurred() == nullptr;
}

template <typename T>
bool convert(PyObject* o, T** out)
{
    void* p;
    if (!address(o, &p)) return false;
    *out = static_cast<T*>(p);
    return true;
}
bool convert(PyObject* o, int* out)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred() != nullptr) return false;
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_SetString(PyExc_OverflowError, "an integer argument does not fit in 32 bits");
        return false;
    }
    *out = static_cast<int>(v);
    return true;
}
bool convert(PyObject* o, float* out)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred() != nullptr) return false;
    *out = static_cast<float>(v);
    return true;
}

// The call of one entry point: all its arguments in order, gives its status.
template <auto Fn>
struct Entry;
template <typename... A, int (*Fn)(A...)>
struct Entry<Fn> {
    template <size_t... I>
    static bool fill(std::tuple<A...>& v, PyObject* const* args, std::index_sequence<I...>)
    {
        return (convert(args[I], &std::get<I>(v)) && ...);
    }
    static PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n)
    {
        if (n != static_cast<Py_ssize_t>(sizeof...(A)))
            return PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given",
                                static_cast<Py_ssize_t>(sizeof...(A)), n);
        std::tuple<A...> v;
        if (!fill(v, args, std::index_sequence_for<A...>{})) return nullptr;
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = std::apply(Fn, v);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(status);
    }
};

template <auto Fn>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&Entry<Fn>::call)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<kv_cache_append>("kv_cache_append"),
    method<bsk_kv_cache_append_enqueue>("bsk_kv_cache_append_enqueue"),
    method<kv_cache_gather>("kv_cache_gather"),
    method<bsk_kv_cache_gather_enqueue>("bsk_kv_cache_gather_enqueue"),
    method<chunk_attention>("chunk_attention"),
    method<bsk_chunk_attention_enqueue>("bsk_chunk_attention_enqueue"),
    method<decode_attention>("decode_attention"),
    method<bsk_decode_attention_enqueue>("bsk_decode_attention_enqueue"),
    method<linear_act>("linear_act"),
    method<bsk_linear_act_enqueue>("bsk_linear_act_enqueue"),
    method<gated_linear>("gated_linear"),
    method<bsk_gated_linear_enqueue>("bsk_gated_linear_enqueue"),
    method<linear_act_backward>("linear_act_backward"),
    method<bsk_linear_act_backward_enqueue>("bsk_linear_act_backward_enqueue"),
    method<gated_linear_backward>("gated_linear_backward"),
    method<bsk_gated_linear_backward_enqueue>("bsk_gated_linear_backward_enqueue"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls()
{
    g_data_ptr = PyUnicode_InternFromString("data_ptr");
    g_ctypes = PyUnicode_InternFromString("ctypes");
    g_data = PyUnicode_InternFromString("data");
    if (g_data_ptr == nullptr || g_ctypes == nullptr || g_data == nullptr) return nullptr;
    return PyModule_Create(&g_module);
}
