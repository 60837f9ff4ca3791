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

#include <pybind11/gil.h>

#include <optional>
#include <utility>

namespace {

constexpr int MOST = 8;               // tensors per call
constexpr at::ScalarType TYPES[] = {at::kFloat, at::kHalf, at::kBFloat16, at::kInt};

PyObject* make(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n < 1 || n % 3 != 1) {
        PyErr_SetString(PyExc_TypeError, "new(device, [type, rows, columns]...)");
        return nullptr;
    }
    const Py_ssize_t count = n / 3;
    if (count > MOST) {
        PyErr_Format(PyExc_TypeError, "at most %d tensors", MOST);
        return nullptr;
    }
    const long index = PyLong_AsLong(args[0]);
    long types[MOST];
    int64_t sizes[MOST][2];
    for (Py_ssize_t i = 0; i < count; ++i) {
        types[i] = PyLong_AsLong(args[3 * i + 1]);
        for (int k = 0; k < 2; ++k) sizes[i][k] = PyLong_AsLongLong(args[3 * i + 2 + k]);
        if (!PyErr_Occurred() && (types[i] < 0 || types[i] > 3))
            PyErr_SetString(PyExc_ValueError, "no such type");
        if (PyErr_Occurred()) return nullptr;
    }
    if (PyErr_Occurred()) return nullptr;
    const at::Device device(at::kCUDA, static_cast<at::DeviceIndex>(index));
    at::Tensor made[MOST];
    {
        // an allocation may wait for the device, whose callbacks may wait for Python
        pybind11::gil_scoped_release released;
        for (Py_ssize_t i = 0; i < count; ++i)
            made[i] = at::detail::empty_cuda(at::IntArrayRef(sizes[i], sizes[i][1] < 0 ? 1 : 2),
                                             TYPES[types[i]], device, std::nullopt);
    }
    PyObject* all = PyTuple_New(count);
    for (Py_ssize_t i = 0; all && i < count; ++i) {
        PyObject* one = THPVariable_Wrap(std::move(made[i]));
        if (one) PyTuple_SET_ITEM(all, i, one);
        else Py_CLEAR(all);
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
