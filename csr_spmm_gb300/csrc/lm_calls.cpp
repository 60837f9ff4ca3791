// The language-model entry points of csr_spmm.h as a Python module, for calls of a few
// microseconds: bind(addresses) takes the loaded library's functions, in the order of
// METHODS, and each function converts its arguments by the C signature (addresses as ints,
// 0 or None for null) and returns the status.
#include <Python.h>

#include <cstddef>
#include <tuple>
#include <type_traits>
#include <utility>

#include "csr_spmm.h"

namespace {

template <typename A>
bool convert(PyObject* o, A& a) {
    if constexpr (std::is_floating_point_v<A>) {
        a = static_cast<A>(PyFloat_AsDouble(o));
    } else if constexpr (std::is_pointer_v<A>) {
        a = o == Py_None ? nullptr : static_cast<A>(PyLong_AsVoidPtr(o));
    } else {
        a = static_cast<A>(PyLong_AsLongLong(o));
    }
    return !PyErr_Occurred();
}

template <int ID, typename F>
struct Entry;
template <int ID, typename... A>
struct Entry<ID, spmm_status_t(A...)> {
    static inline spmm_status_t (*fn)(A...) = nullptr;

    static PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
        if (n != sizeof...(A)) {
            PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", (int)sizeof...(A), n);
            return nullptr;
        }
        if (!fn) {
            PyErr_SetString(PyExc_RuntimeError, "bind the library's functions first");
            return nullptr;
        }
        return call_with(args, std::index_sequence_for<A...>{});
    }
    template <size_t... I>
    static PyObject* call_with(PyObject* const* args, std::index_sequence<I...>) {
        std::tuple<A...> a;
        if (!(convert(args[I], std::get<I>(a)) && ...)) return nullptr;
        spmm_status_t status;
        Py_BEGIN_ALLOW_THREADS
        status = fn(std::get<I>(a)...);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(static_cast<long>(status));
    }
};

using Embedding = Entry<0, decltype(spmm_embedding)>;
using EmbeddingGrad = Entry<1, decltype(spmm_embedding_grad)>;
using LayerNorm = Entry<2, decltype(spmm_layer_norm)>;
using LayerNormGrad = Entry<3, decltype(spmm_layer_norm_grad)>;
using TokenLogprob = Entry<4, decltype(spmm_token_logprob)>;
using TokenLogprobGrad = Entry<5, decltype(spmm_token_logprob_grad)>;

template <typename E>
void set(void* address) {
    E::fn = reinterpret_cast<decltype(E::fn)>(address);
}

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "six addresses expected");
        return nullptr;
    }
    void* address[6];
    for (int i = 0; i < 6; ++i)
        if (!convert(args[i], address[i])) return nullptr;
    set<Embedding>(address[0]);
    set<EmbeddingGrad>(address[1]);
    set<LayerNorm>(address[2]);
    set<LayerNormGrad>(address[3]);
    set<TokenLogprob>(address[4]);
    set<TokenLogprobGrad>(address[5]);
    Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL,
            nullptr};
}
PyMethodDef METHODS[] = {method("spmm_embedding", Embedding::call),
                         method("spmm_embedding_grad", EmbeddingGrad::call),
                         method("spmm_layer_norm", LayerNorm::call),
                         method("spmm_layer_norm_grad", LayerNormGrad::call),
                         method("spmm_token_logprob", TokenLogprob::call),
                         method("spmm_token_logprob_grad", TokenLogprobGrad::call),
                         method("bind", bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef MODULE = {PyModuleDef_HEAD_INIT, "_lm_calls", nullptr, -1, METHODS,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm_calls() { return PyModule_Create(&MODULE); }
