// host_checks.cpp -- the binding's argument checks, natively.
//
// A call on a few tokens is bound by the host.  Of 7.0 us a call with four
// tensors the launch took 3.4 and the checks' way through the interpreter most
// of the rest (0.3 us a tensor for dtype, layout and shape, 0.14 for its
// device, 0.09 for its pointer; 0.27 us a tensor and list for lists of
// gradients); with this module a call takes 4.5.  It answers the usual case, a
// plain strided tensor that fits, from the tensor itself; whatever else it is
// given goes to the Python function of the same name, which decides and
// raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

PyObject *g_check_arg, *g_check_device, *g_ptr;   // the Python functions

// The tensor behind o, where it is a plain strided one; else nullptr.
const at::Tensor* plain(PyObject* o) {
    if (!THPVariable_CheckTypeExact(Py_TYPE(o))) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.defined() && t.layout() == at::kStrided ? &t : nullptr;
}

int64_t current_device() {
    return c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index();
}

// As check_arg, without its errors: whether t is known to fit.
bool fits(PyObject* o, PyObject* dtypes, PyObject* shape, PyObject* min_rows) {
    const at::Tensor* t = plain(o);
    if (!t || !PyTuple_Check(dtypes) || !t->is_contiguous()) return false;
    bool type = false;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(dtypes) && !type; ++i) {
        PyObject* d = PyTuple_GET_ITEM(dtypes, i);
        type = THPDtype_Check(d) && reinterpret_cast<THPDtype*>(d)->scalar_type == t->scalar_type();
    }
    if (!type) return false;
    if (shape == Py_None) return true;
    if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t->dim()) return false;
    for (Py_ssize_t i = 0; i < t->dim(); ++i) {
        PyObject* want = i == 0 && min_rows != Py_None ? min_rows : PyTuple_GET_ITEM(shape, i);
        if (want == Py_None) continue;
        if (!PyLong_Check(want)) return false;
        const long long w = PyLong_AsLongLong(want);
        if (w == -1 && PyErr_Occurred()) return false;
        if (want == min_rows && i == 0 ? t->size(i) < w : t->size(i) != w) return false;
    }
    return true;
}

// check_arg(t, name, dtypes, shape=None, min_rows=None, optional=False)
PyObject* check_arg(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* names) {
    PyObject* opt[3] = {Py_None, Py_None, Py_False};   // shape, min_rows, optional
    static const char* const kNames[3] = {"shape", "min_rows", "optional"};
    bool usual = n >= 3 && n <= 6;
    for (Py_ssize_t i = 3; usual && i < n; ++i) opt[i - 3] = args[i];
    for (Py_ssize_t k = 0; usual && names && k < PyTuple_GET_SIZE(names); ++k) {
        int j = 0;
        while (j < 3 && PyUnicode_CompareWithASCIIString(PyTuple_GET_ITEM(names, k), kNames[j]) != 0) ++j;
        if (j == 3 || j + 3 < n) usual = false;   // unknown, or given by place as well
        else opt[j] = args[n + k];
    }
    if (usual) {
        try {
            if (args[0] == Py_None ? opt[2] == Py_True : fits(args[0], args[2], opt[0], opt[1])) Py_RETURN_NONE;
        } catch (...) {
        }
        PyErr_Clear();
    }
    return PyObject_Vectorcall(g_check_arg, args, n, names);
}

// check_device(*tensors)
PyObject* check_device(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        int64_t current = -1;
        Py_ssize_t i = 0;
        for (; i < n; ++i) {
            if (args[i] == Py_None) continue;
            const at::Tensor* t = plain(args[i]);
            if (!t || !t->is_cuda()) break;
            if (current < 0) current = current_device();
            if (t->device().index() != current) break;
        }
        if (i == n) Py_RETURN_NONE;
    } catch (...) {
    }
    PyErr_Clear();
    return PyObject_Vectorcall(g_check_device, args, n, nullptr);
}

// ptr(t): its data pointer, None for None
PyObject* ptr(PyObject*, PyObject* o) {
    if (o == Py_None) Py_RETURN_NONE;
    try {
        if (const at::Tensor* t = plain(o)) return PyLong_FromVoidPtr(t->data_ptr());
    } catch (...) {
    }
    PyErr_Clear();
    return PyObject_CallFunctionObjArgs(g_ptr, o, nullptr);
}

// A tensor of a gradient list: whether it is usual, and its kind (0 bf16 or
// its bits, 1 fp32).
bool grad(PyObject* o, int64_t current, const at::Tensor*& t, int64_t& kind) {
    t = plain(o);
    if (!t || !t->is_cuda() || t->device().index() != current || !t->is_contiguous()) return false;
    const at::ScalarType s = t->scalar_type();
    kind = s == at::kFloat ? 1 : 0;
    return kind == 1 || s == at::kBFloat16 || s == at::kShort;
}

// grad_words(grads, outs): the moe_grad_tensor array of two lists (which may
// be one) as bytes, or None where a tensor is unusual or does not fit.
PyObject* grad_words(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 2 || !PyList_Check(args[0]) || !PyList_Check(args[1])) Py_RETURN_NONE;
    const Py_ssize_t num = PyList_GET_SIZE(args[0]);
    if (PyList_GET_SIZE(args[1]) != num || num == 0) Py_RETURN_NONE;
    PyObject* bytes = PyBytes_FromStringAndSize(nullptr, num * 32);
    if (!bytes) return nullptr;
    uint64_t* w = reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(bytes));
    bool usual = true;
    try {
        const int64_t current = plain(PyList_GET_ITEM(args[0], 0)) ? current_device() : -1;
        for (Py_ssize_t i = 0; i < num && usual; ++i, w += 4) {
            PyObject *go = PyList_GET_ITEM(args[0], i), *oo = PyList_GET_ITEM(args[1], i);
            const at::Tensor *g, *o;
            int64_t kg, ko;
            usual = grad(go, current, g, kg);
            if (!usual) break;
            o = g;
            ko = kg;
            if (oo != go) usual = grad(oo, current, o, ko) && ko == kg && o->numel() == g->numel();
            if (!usual) break;
            w[0] = reinterpret_cast<uintptr_t>(g->data_ptr());
            w[1] = reinterpret_cast<uintptr_t>(o->data_ptr());
            w[2] = (uint64_t)g->numel();
            w[3] = (uint64_t)kg;
        }
    } catch (...) {
        usual = false;
    }
    PyErr_Clear();
    if (usual) return bytes;
    Py_DECREF(bytes);
    Py_RETURN_NONE;
}

// bind(check_arg, check_device, ptr): the Python functions
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "bind takes three functions");
        return nullptr;
    }
    PyObject** const to[3] = {&g_check_arg, &g_check_device, &g_ptr};
    for (int i = 0; i < 3; ++i) {
        Py_INCREF(args[i]);
        Py_XDECREF(*to[i]);
        *to[i] = args[i];
    }
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef kMethods[] = {{"check_arg", FAST(check_arg), METH_FASTCALL | METH_KEYWORDS, nullptr},
                          {"check_device", FAST(check_device), METH_FASTCALL, nullptr},
                          {"ptr", ptr, METH_O, nullptr},
                          {"grad_words", FAST(grad_words), METH_FASTCALL, nullptr},
                          {"bind", FAST(bind), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__host() { return PyModule_Create(&kModule); }
