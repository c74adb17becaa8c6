// Tensor arguments of the round calls, checked and taken apart natively: the binding spends about a tenth of a
// microsecond on a tensor here, half of one in Python, and a small call has up to fifteen of them.  Nothing of the
// C ABI library is used, and the library uses nothing of this.
//
//   ptr(tensor, name, dtype, shape, device)   its address
//   opt(tensor or None, ...)                  the same, or None
//   view(tensor, name, dtype, shape, device)  a gdn_heads_view of a [C, N, heads, D] tensor as bytes
//   init(refuse)                              before these: refuse(tensor, name, dtype, shape, device) is called with a
//                                             tensor of another type, shape, device or layout, and raises
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

PyObject *g_refuse = nullptr;

// The tensor where it has this dtype, shape and device; else nullptr with the error of refuse() set.
const at::Tensor *checked(PyObject *const *a, Py_ssize_t n, bool contiguous) {
    if (!g_refuse || n != 5 || !THPDtype_Check(a[2]) || !PyTuple_Check(a[3])) {
        PyErr_SetString(PyExc_TypeError, "expected (tensor, name, dtype, shape, device), after init(refuse)");
        return nullptr;
    }
    const long device = PyLong_AsLong(a[4]);
    if (device == -1 && PyErr_Occurred()) return nullptr;
    if (THPVariable_Check(a[0])) {
        const at::Tensor &t = THPVariable_Unpack(a[0]);
        const Py_ssize_t dims = PyTuple_GET_SIZE(a[3]);
        bool same = t.scalar_type() == reinterpret_cast<THPDtype *>(a[2])->scalar_type && t.dim() == dims &&
                    t.is_cuda() && t.get_device() == device && t.layout() == at::kStrided;
        for (Py_ssize_t k = 0; same && k < dims; ++k) {
            const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(a[3], k));
            if (want == -1 && PyErr_Occurred()) return nullptr;
            same = t.size(k) == want;
        }
        if (same && (!contiguous || t.is_contiguous())) return &t;
    }
    PyObject *r = PyObject_CallFunctionObjArgs(g_refuse, a[0], a[1], a[2], a[3], a[4], nullptr);
    if (r) {
        Py_DECREF(r);
        PyErr_SetString(PyExc_ValueError, "unsuitable tensor");
    }
    return nullptr;
}

PyObject *ptr(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS  // (a tensor without storage or with symbolic sizes throws)
    const at::Tensor *t = checked(a, n, true);
    return t ? PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t->data_ptr())) : nullptr;
    END_HANDLE_TH_ERRORS
}

PyObject *opt(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (n == 5 && a[0] == Py_None) Py_RETURN_NONE;
    return ptr(self, a, n);
}

PyObject *view(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *t = checked(a, n, false);
    if (!t) return nullptr;
    if (t->dim() != 4) {
        PyErr_SetString(PyExc_TypeError, "a view has four dimensions");
        return nullptr;
    }
    const int64_t C = t->size(0), N = t->size(1), heads = t->size(2);
    if (t->size(3) > 1 && t->stride(3) != 1) {
        PyErr_Format(PyExc_ValueError, "%U: values of one head must be contiguous", a[1]);
        return nullptr;
    }
    if (N > 1 && C > 1 && t->stride(0) != N * t->stride(1)) {
        PyErr_Format(PyExc_ValueError, "%U: token rows must be evenly strided across lanes", a[1]);
        return nullptr;
    }
    const int64_t v[3] = {static_cast<int64_t>(reinterpret_cast<uintptr_t>(t->data_ptr())),
                          N > 1 ? t->stride(1) : C > 1 ? t->stride(0) : 0, heads > 1 ? t->stride(2) : 0};
    return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(v), sizeof v);
    END_HANDLE_TH_ERRORS
}

PyObject *init(PyObject *, PyObject *refuse) {
    Py_INCREF(refuse);
    Py_XSETREF(g_refuse, refuse);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_O, "the function that raises for an unsuitable tensor"},
    {"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(ptr)), METH_FASTCALL, "address of a checked tensor"},
    {"opt", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(opt)), METH_FASTCALL, "the same, None for None"},
    {"view", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(view)), METH_FASTCALL, "a gdn_heads_view as bytes"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "checked tensor arguments of the round calls", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
