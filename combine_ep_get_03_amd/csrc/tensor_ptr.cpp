// tensor_ptr.cpp -- the Python module _tensor_ptr: one tensor argument of a call checked and
// turned into its device address. Host code only; the binding of the calls themselves is
// ctypes over libep.so.
//
//   row_ptr(tensor, dtype, shape, name, device, need=True) -> int or None
//   dims2(tensor, name) -> (rows, columns)
//
// row_ptr: the address of a dense tensor of exactly this type and shape (None: any shape of
// one element or more) on this device; None for None unless it is needed. dims2: the sizes of
// a tensor of two dimensions. Anything else goes to the callable given to set_explain, which
// raises, with the same arguments but the device (from dims2 with None for what it does not
// have). A check costs 0.1 us here and 0.43 us as five attribute and method calls in Python,
// and a call of the norm makes eight of them.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

namespace {

PyObject* explain = nullptr;

PyObject* complain(PyObject* tensor, PyObject* dtype, PyObject* shape, PyObject* name,
                   PyObject* need) {
    if (!explain) {
        PyErr_SetString(PyExc_RuntimeError, "_tensor_ptr: set_explain has not been called");
        return nullptr;
    }
    PyObject* r = PyObject_CallFunctionObjArgs(explain, tensor, dtype, shape, name, need, nullptr);
    if (!r) return nullptr;
    Py_DECREF(r);
    PyErr_Format(PyExc_ValueError, "%S is not a tensor that this call takes", name);
    return nullptr;
}

// 1 if the tensor has exactly this shape, 0 if not, -1 with a Python error set.
int same_shape(const at::Tensor& t, PyObject* shape) {
    if (shape == Py_None) return t.numel() >= 1;
    if (!PyTuple_Check(shape)) return 0;
    const Py_ssize_t n = PyTuple_GET_SIZE(shape);
    if (n != t.dim()) return 0;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const long long d = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
        if (d == -1 && PyErr_Occurred()) return -1;
        if (d != t.size(i)) return 0;
    }
    return 1;
}

PyObject* row_ptr(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5 && n != 6) {
        PyErr_SetString(PyExc_TypeError, "row_ptr(tensor, dtype, shape, name, device, need=True)");
        return nullptr;
    }
    PyObject* need = n == 6 ? a[5] : Py_True;
    if (a[0] == Py_None && need != Py_True) Py_RETURN_NONE;
    if (!THPVariable_Check(a[0]) || !THPDtype_Check(a[1]))
        return complain(a[0], a[1], a[2], a[3], need);
    const long device = PyLong_AsLong(a[4]);
    if (device == -1 && PyErr_Occurred()) return nullptr;
    try {  // a tensor without plain storage (sparse, fake) throws on some of these
        const at::Tensor& t = THPVariable_Unpack(a[0]);
        const bool ok = t.is_cuda() &&
                        t.scalar_type() == reinterpret_cast<THPDtype*>(a[1])->scalar_type &&
                        t.get_device() == device && t.is_contiguous();
        const int shape = ok ? same_shape(t, a[2]) : 0;
        if (shape < 0) return nullptr;
        if (shape == 1) return PyLong_FromVoidPtr(t.data_ptr());
    } catch (const std::exception&) {
    }
    return complain(a[0], a[1], a[2], a[3], need);
}

PyObject* dims2(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "dims2(tensor, name)");
        return nullptr;
    }
    if (THPVariable_Check(a[0])) {
        try {
            const at::Tensor& t = THPVariable_Unpack(a[0]);
            if (t.dim() == 2)
                return Py_BuildValue("(LL)", static_cast<long long>(t.size(0)),
                                     static_cast<long long>(t.size(1)));
        } catch (const std::exception&) {
        }
    }
    return complain(a[0], Py_None, Py_None, a[1], Py_True);
}

PyObject* set_explain(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XSETREF(explain, f);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"row_ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(row_ptr)),
     METH_FASTCALL, "row_ptr(tensor, dtype, shape, name, device, need=True) -> int or None"},
    {"dims2", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dims2)), METH_FASTCALL,
     "dims2(tensor, name) -> (rows, columns)"},
    {"set_explain", set_explain, METH_O, "the callable that refuses a tensor"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_ptr", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_ptr() { return PyModule_Create(&module); }
