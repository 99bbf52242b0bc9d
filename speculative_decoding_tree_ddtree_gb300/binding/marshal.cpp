// marshal.cpp -- the tensor check of the Python binding in one C call.
//
// A call of a small step is bound by the host, and reading a tensor's type, shape,
// device, contiguity and address through Python attributes costs about 0.4 us a
// tensor (measured on the GPU machine): arg() makes the same checks on the tensor
// itself; whatever it does not find in order goes to the Python function that
// set_slow() names, which raises the error that says why.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

namespace {

constexpr int kKinds = 8;
PyObject* g_slow = nullptr;
unsigned long long g_types[kKinds] = {};  // bit t: element type t is fine; 0: any type
int g_kinds = 0;

// Address of a contiguous tensor of this kind on device `dev` (-1: host), of the given
// sizes (none given: any, but not empty); false if anything is different.
bool address_of(PyObject* obj, long kind, long dev, PyObject* const* sizes, Py_ssize_t n, unsigned long long* out) {
    if (!THPVariable_Check(obj) || kind < 0 || kind >= g_kinds) return false;
    const at::Tensor& t = THPVariable_Unpack(obj);
    if (!t.defined() || t.layout() != at::kStrided) return false;
    if (g_types[kind] && !((g_types[kind] >> (int)t.scalar_type()) & 1ull)) return false;
    if (dev >= 0 ? !(t.is_cuda() && t.get_device() == dev) : !t.is_cpu()) return false;
    if (n == 0) {
        if (t.numel() == 0) return false;
    } else {
        if (t.dim() != n) return false;
        for (Py_ssize_t i = 0; i < n; ++i) {
            const long long want = PyLong_AsLongLong(sizes[i]);
            if (want < 0 || t.size(i) != want) return false;  // (-1 is also the error value)
        }
    }
    if (!t.is_contiguous()) return false;
    *out = (unsigned long long)reinterpret_cast<uintptr_t>(t.data_ptr());
    return true;
}

// arg(tensor, name, kind, dev, *sizes)
PyObject* arg(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n >= 4 && g_slow) {
        const long kind = PyLong_AsLong(a[2]), dev = PyLong_AsLong(a[3]);
        unsigned long long at = 0;
        bool ok = false;
        if (!PyErr_Occurred()) {
            try {
                ok = address_of(a[0], kind, dev, a + 4, n - 4, &at);
            } catch (...) {  // a tensor without plain data: the slow path says so
            }
        }
        if (ok && !PyErr_Occurred()) return PyLong_FromUnsignedLongLong(at);
        PyErr_Clear();
        return PyObject_Vectorcall(g_slow, a, (size_t)n, nullptr);
    }
    PyErr_SetString(PyExc_TypeError, "arg(tensor, name, kind, dev, *sizes) after set_slow()");
    return nullptr;
}

// set_slow(function, [one example dtype tuple's bit mask per kind])
PyObject* set_slow(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 2 || !PyCallable_Check(a[0]) || !PyList_Check(a[1]) || PyList_GET_SIZE(a[1]) > kKinds) {
        PyErr_SetString(PyExc_TypeError, "set_slow(function, masks)");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(a[1]); ++i) {
        g_types[i] = PyLong_AsUnsignedLongLong(PyList_GET_ITEM(a[1], i));
        if (PyErr_Occurred()) return nullptr;
    }
    g_kinds = (int)PyList_GET_SIZE(a[1]);
    Py_INCREF(a[0]);
    Py_XDECREF(g_slow);
    g_slow = a[0];
    Py_RETURN_NONE;
}

// Number of a tensor's element type, for the masks.
PyObject* type_of(PyObject*, PyObject* obj) {
    if (!THPVariable_Check(obj)) {
        PyErr_SetString(PyExc_TypeError, "type_of(tensor)");
        return nullptr;
    }
    return PyLong_FromLong((long)THPVariable_Unpack(obj).scalar_type());
}

PyMethodDef kMethods[] = {
    {"arg", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(arg)), METH_FASTCALL, nullptr},
    {"set_slow", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(set_slow)), METH_FASTCALL, nullptr},
    {"type_of", type_of, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject* m = PyModule_Create(&kModule);
    if (m && PyModule_AddStringConstant(m, "torch_version", MARSHAL_TORCH_VERSION) != 0) Py_CLEAR(m);
    return m;
}
