// Output tensors for small calls, as a Python module: new(device, type, rows, columns,
// type, rows, columns, ...) gives a tuple of uninitialised CUDA tensors on torch's current
// stream of that device (columns < 0: a vector of `rows`; type 0 to 2: spmm_type_t, 3:
// int32).  The memory comes from torch's caching allocator, as torch.empty's does, without
// torch.empty's argument parsing and dispatch for each.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <optional>

namespace {

constexpr at::ScalarType TYPES[] = {at::kFloat, at::kHalf, at::kBFloat16, at::kInt};

PyObject* make(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n < 1 || n % 3 != 1) {
        PyErr_SetString(PyExc_TypeError, "new(device, [type, rows, columns]...)");
        return nullptr;
    }
    const at::Device device(at::kCUDA, static_cast<at::DeviceIndex>(PyLong_AsLong(args[0])));
    PyObject* all = PyTuple_New(n / 3);
    if (!all) return nullptr;
    for (Py_ssize_t i = 0; i < n / 3; ++i) {
        const long type = PyLong_AsLong(args[3 * i + 1]);
        const std::array<int64_t, 2> sizes{PyLong_AsLongLong(args[3 * i + 2]),
                                           PyLong_AsLongLong(args[3 * i + 3])};
        if (PyErr_Occurred() || type < 0 || type > 3) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no such type");
            Py_DECREF(all);
            return nullptr;
        }
        at::Tensor t;
        try {
            t = at::detail::empty_cuda(at::IntArrayRef(sizes.data(), sizes[1] < 0 ? 1 : 2),
                                       TYPES[type], device, std::nullopt);
        } catch (...) {
            Py_DECREF(all);
            throw;
        }
        PyObject* one = THPVariable_Wrap(std::move(t));
        if (!one) {
            Py_DECREF(all);
            return nullptr;
        }
        PyTuple_SET_ITEM(all, i, one);
    }
    return all;
    END_HANDLE_TH_ERRORS
}

PyMethodDef METHODS[] = {
    {"new", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(make)), METH_FASTCALL,
     "Uninitialised CUDA tensors: new(device, [type, rows, columns]...)."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef MODULE = {PyModuleDef_HEAD_INIT, "_torch_outputs", nullptr, -1, METHODS,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_outputs() { return PyModule_Create(&MODULE); }
