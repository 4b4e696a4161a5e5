// The binding's check of one tensor argument, as a Python extension:
//
//   arg(tensor, name, dtype, shape, device) -> int
//   opt(...)                                -> int, or None for None
//
// the tensor's data address if it is a contiguous tensor of that dtype and shape
// (a tuple) on that CUDA device index; otherwise the Python function given to
// refuse_with() is called with (tensor, name, dtype, shape) to raise the error.
// The calls of a decode step run for a few microseconds on the GPU, and the same
// attribute reads in Python take about 0.5 us a tensor (here about 0.1), so that
// a call with five tensors waited for its checks.  Nothing is kept of a tensor.
// torch_version names the torch that it was compiled against: the binding makes the
// checks in Python where that is not the running one, or where this is not built.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <Python.h>

namespace {

PyObject* g_refuse = nullptr;

// 1: the tensor is as asked, 0: it is not, -1: a Python error is set
int as_asked(PyObject* tensor, PyObject* dtype, PyObject* shape, PyObject* device, void** address) {
    if (!THPVariable_Check(tensor) || !THPDtype_Check(dtype) || !PyTuple_Check(shape)) return 0;
    const long dev = PyLong_AsLong(device);
    if (dev == -1 && PyErr_Occurred()) return -1;
    const at::Tensor& t = THPVariable_Unpack(tensor);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type)
        return 0;
    const Py_ssize_t dims = PyTuple_GET_SIZE(shape);
    if (t.dim() != dims) return 0;
    const c10::IntArrayRef sizes = t.sizes();
    for (Py_ssize_t i = 0; i < dims; ++i) {
        const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
        if (want == -1 && PyErr_Occurred()) return -1;
        if (sizes[i] != want) return 0;
    }
    if (!t.is_contiguous()) return 0;
    *address = t.data_ptr();
    return 1;
}

PyObject* arg(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "arg(tensor, name, dtype, shape, device)");
        return nullptr;
    }
    try {
        void* address = nullptr;
        const int ok = as_asked(a[0], a[2], a[3], a[4], &address);
        if (ok < 0) return nullptr;
        if (ok) return PyLong_FromVoidPtr(address);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    PyObject* r = g_refuse ? PyObject_CallFunctionObjArgs(g_refuse, a[0], a[1], a[2], a[3], nullptr) : nullptr;
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "tensor argument refused");
    return nullptr;
}

PyObject* opt(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n == 5 && a[0] == Py_None) Py_RETURN_NONE;
    return arg(self, a, n);
}

PyObject* refuse_with(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XSETREF(g_refuse, f);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F* f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {
    {"arg", method(arg), METH_FASTCALL, nullptr},
    {"opt", method(opt), METH_FASTCALL, nullptr},
    {"refuse_with", refuse_with, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycheck", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycheck() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
