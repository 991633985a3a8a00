// The binding's checks of the tensors it is given, for the usual call: a Python module of two functions that look at a
// tensor's type, device, shape and strides where torch holds them, and hand out addresses. Anything that is not as the
// kernels take it gives None, and the binding's own checks then say what is wrong. (A call's tensors on 8 ranks cost 0.4 to 0.5 us each
// when Python looked at them.)
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// A tensor shape or number of elements as the caller gives it.
struct Shape {
    bool flat = false;  // a number of elements, of any shape
    int64_t numel = 0;
    int dims = 0;
    int64_t size[4];
};

bool read_shape(PyObject* o, Shape* s) {
    if (PyLong_Check(o)) {
        s->flat = true;
        s->numel = PyLong_AsLongLong(o);
        return !PyErr_Occurred();
    }
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) > 4) return false;
    s->dims = int(PyTuple_GET_SIZE(o));
    for (int i = 0; i < s->dims; ++i) {
        s->size[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        if (s->size[i] == -1 && PyErr_Occurred()) return false;
    }
    return true;
}

// The address of a tensor that is as asked: contiguous, or, with ld >= 0, rows of one dimension at that distance.
bool address_of(PyObject* o, at::ScalarType type, const Shape& s, long device, int64_t ld, void** to) {
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || t.scalar_type() != type) return false;
    if (t.is_cuda() ? t.get_device() != device : !(t.is_cpu() && device == -1)) return false;
    if (s.flat) {
        if (t.numel() != s.numel) return false;
    } else {
        const auto sizes = t.sizes();
        if (int(sizes.size()) != s.dims) return false;
        for (int i = 0; i < s.dims; ++i)
            if (sizes[i] != s.size[i]) return false;
    }
    if (ld >= 0 && !s.flat && s.dims == 2 && s.size[0] > 1) {
        if (t.stride(1) != 1 || t.stride(0) != ld) return false;
    } else if (!t.is_contiguous()) {
        return false;
    }
    *to = t.data_ptr();
    return true;
}

// addresses(tensors, dtype, shape, device, ranks, ld) -> bytes of `ranks` pointers, or None
PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 6 || !THPDtype_Check(args[1])) Py_RETURN_NONE;
    const long device = PyLong_AsLong(args[3]), ranks = PyLong_AsLong(args[4]);
    const int64_t ld = PyLong_AsLongLong(args[5]);
    Shape s;
    void* found[64];
    const bool list = PyList_Check(args[0]);
    if (PyErr_Occurred() || !read_shape(args[2], &s) || !(list || PyTuple_Check(args[0])) || ranks < 1 || ranks > 64 ||
        (list ? PyList_GET_SIZE(args[0]) : PyTuple_GET_SIZE(args[0])) != ranks) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const at::ScalarType type = reinterpret_cast<THPDtype*>(args[1])->scalar_type;
    try {
        for (long r = 0; r < ranks; ++r) {
            PyObject* t = list ? PyList_GET_ITEM(args[0], r) : PyTuple_GET_ITEM(args[0], r);
            if (!address_of(t, type, s, device, ld, &found[r])) Py_RETURN_NONE;
        }
    } catch (...) {  // a tensor without memory
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(found), Py_ssize_t(ranks * sizeof(void*)));
}

// address(tensor, dtype, shape, device) -> the address, or None
PyObject* address(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 4 || !THPDtype_Check(args[1])) Py_RETURN_NONE;
    const long device = PyLong_AsLong(args[3]);
    Shape s;
    void* found = nullptr;
    if (PyErr_Occurred() || !read_shape(args[2], &s)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    try {
        if (!address_of(args[0], reinterpret_cast<THPDtype*>(args[1])->scalar_type, s, device, -1, &found)) Py_RETURN_NONE;
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    return PyLong_FromVoidPtr(found);
}

PyMethodDef methods[] = {
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(addresses)), METH_FASTCALL,
     "addresses(tensors, dtype, shape, device, ranks, ld): the bytes of the tensors' addresses, or None"},
    {"address", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(address)), METH_FASTCALL,
     "address(tensor, dtype, shape, device): the tensor's address, or None"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Addresses of checked tensors.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
