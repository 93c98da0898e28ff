// The argument checks of the Python binding's calls, natively: what they cost in
// Python is more than a small call's launch (four tensors: 2.0 us there, 0.3
// here).  Whatever is not in order is handed to the Python method of the same
// purpose, which says what is wrong; nothing is refused here alone.
//
// Tensors are read by torch's inline accessors, whose offsets are those of the
// torch that this was built for.  With another one the import fails, and the
// binding checks in Python.
#include <Python.h>
#include <structmember.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>
#include <torch/csrc/utils/tensor_dtypes.h>

namespace {

constexpr int kMaxArgs = 24;

struct Entry {
    uintptr_t at, end;
    PyObject* name;
    PyObject* tensor;
    int device;  // -1: none of the GPUs
    bool written;
};

struct Checks {
    PyObject_HEAD
    PyObject* call;     // name of the C entry point
    PyObject* tensors;  // list of the Python methods
    int count;
    Entry entries[kMaxArgs];
};

PyObject* raw_stream = nullptr;  // index of a GPU -> handle of its current stream

PyObject* checks_new(PyTypeObject* type, PyObject*, PyObject*) {
    auto* self = reinterpret_cast<Checks*>(type->tp_alloc(type, 0));
    if (!self) return nullptr;
    self->tensors = PyList_New(0);
    if (!self->tensors) {
        Py_DECREF(self);
        return nullptr;
    }
    return reinterpret_cast<PyObject*>(self);
}

int checks_init(PyObject* o, PyObject* args, PyObject*) {
    auto* self = reinterpret_cast<Checks*>(o);
    PyObject* call;
    if (!PyArg_UnpackTuple(args, "Checks", 1, 1, &call)) return -1;
    Py_INCREF(call);
    Py_XSETREF(self->call, call);
    return 0;
}

void checks_dealloc(PyObject* o) {
    auto* self = reinterpret_cast<Checks*>(o);
    Py_XDECREF(self->call);
    Py_XDECREF(self->tensors);
    for (int i = 0; i < self->count; ++i) {
        Py_DECREF(self->entries[i].name);
        Py_DECREF(self->entries[i].tensor);
    }
    Py_TYPE(o)->tp_free(o);
}

bool has_type(PyObject* dtypes, PyObject* dtype) {
    if (dtypes == Py_None) return true;
    const Py_ssize_t n = PyTuple_GET_SIZE(dtypes);
    for (Py_ssize_t i = 0; i < n; ++i)
        if (PyTuple_GET_ITEM(dtypes, i) == dtype) return true;
    return false;
}

// arg(name, tensor, dtypes, nbytes, optional=False, written=False): the tensor's address.
PyObject* checks_arg(PyObject* o, PyObject* const* a, Py_ssize_t nargs, PyObject* kwnames) {
    HANDLE_TH_ERRORS  // torch's C++ exceptions become Python's
    auto* self = reinterpret_cast<Checks*>(o);
    const Py_ssize_t nkw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    if (nargs < 4 || nargs + nkw > 6 || (a[2] != Py_None && !PyTuple_Check(a[2]))) {
        PyErr_SetString(PyExc_TypeError, "arg(name, tensor, dtypes, nbytes, optional=False, written=False)");
        return nullptr;
    }
    PyObject* optional = nargs > 4 ? a[4] : Py_False;
    bool written = nargs > 5 && PyObject_IsTrue(a[5]);
    for (Py_ssize_t i = 0; i < nkw; ++i) {
        PyObject* key = PyTuple_GET_ITEM(kwnames, i);
        if (PyUnicode_CompareWithASCIIString(key, "written") == 0) {
            written = PyObject_IsTrue(a[nargs + i]);
        } else if (PyUnicode_CompareWithASCIIString(key, "optional") == 0) {
            optional = a[nargs + i];
        } else {
            PyErr_SetString(PyExc_TypeError, "arg: unexpected keyword");
            return nullptr;
        }
    }
    int overflow;  // sizes of absurd shapes pass 64 bits; no tensor holds that many bytes
    const long long need = PyLong_AsLongLongAndOverflow(a[3], &overflow);
    if (need == -1 && PyErr_Occurred()) return nullptr;
    PyObject* t = a[1];
    bool good = false;
    if (THPVariable_CheckExact(t)) {
        const at::Tensor& v = THPVariable_Unpack(t);
        good = overflow <= 0 && v.layout() == at::kStrided && v.is_contiguous() && (long long)v.nbytes() >= need &&
               has_type(a[2], reinterpret_cast<PyObject*>(torch::getTHPDtype(v.scalar_type())));
    }
    if (!good) {  // a subclass or none, or something to complain of
        PyObject* r = PyObject_CallMethod(o, "need", "OOOOO", a[0], t, a[2], a[3], optional);
        if (!r) return nullptr;
        Py_DECREF(r);
        if (t == Py_None) Py_RETURN_NONE;
    }
    if (!THPVariable_Check(t) || self->count == kMaxArgs) {
        PyErr_SetString(PyExc_TypeError, "arg: no tensor, or too many of them");
        return nullptr;
    }
    const at::Tensor& v = THPVariable_Unpack(t);
    Entry& e = self->entries[self->count];
    e.at = reinterpret_cast<uintptr_t>(v.data_ptr());
    e.end = e.at + v.nbytes();
    e.device = v.is_cuda() ? v.get_device() : -1;
    e.written = written;
    Py_INCREF(a[0]);
    e.name = a[0];
    Py_INCREF(t);
    e.tensor = t;
    ++self->count;
    return PyLong_FromUnsignedLongLong(e.at);
    END_HANDLE_TH_ERRORS
}

// on_device(stream): (the GPU's index, the stream's handle), see binding.py.
PyObject* checks_on_device(PyObject* o, PyObject* stream) {
    auto* self = reinterpret_cast<Checks*>(o);
    const int n = self->count;
    bool good = stream == Py_None && n > 0 && self->entries[0].device >= 0;
    for (int i = 0; i < n && good; ++i) {
        const Entry& e = self->entries[i];
        good = e.device == self->entries[0].device;
        if (e.written)
            for (int j = 0; j < n && good; ++j) {
                const Entry& f = self->entries[j];
                good = j == i || !(e.at < f.end && f.at < e.end);
            }
    }
    if (good) {
        THPObjectPtr dev(PyLong_FromLong(self->entries[0].device));
        if (!dev) return nullptr;
        THPObjectPtr handle(PyObject_CallOneArg(raw_stream, dev.get()));
        if (!handle) return nullptr;
        return PyTuple_Pack(2, dev.get(), handle.get());
    }
    THPObjectPtr lists[2] = {THPObjectPtr(PyList_New(0)), THPObjectPtr(PyList_New(0))};
    for (int i = 0; i < n; ++i) {
        const Entry& e = self->entries[i];
        THPObjectPtr item(Py_BuildValue("(KKOO)", (unsigned long long)e.at, (unsigned long long)e.end, e.name, e.tensor));
        if (!item || !lists[0] || !lists[1] || PyList_Append(lists[e.written ? 1 : 0].get(), item.get()) < 0)
            return nullptr;
    }
    return PyObject_CallMethod(o, "resolve", "OOO", lists[0].get(), lists[1].get(), stream);
}

PyMemberDef members[] = {
    {"call", T_OBJECT_EX, offsetof(Checks, call), 0, nullptr},
    {"tensors", T_OBJECT_EX, offsetof(Checks, tensors), 0, nullptr},
    {nullptr, 0, 0, 0, nullptr},
};

PyMethodDef methods[] = {
    {"arg", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(checks_arg)), METH_FASTCALL | METH_KEYWORDS, nullptr},
    {"on_device", checks_on_device, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyTypeObject type = {PyVarObject_HEAD_INIT(nullptr, 0)};

PyObject* use_stream_of(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XSETREF(raw_stream, f);
    Py_RETURN_NONE;
}

PyMethodDef functions[] = {
    {"use_stream_of", use_stream_of, METH_O, "The function that gives a GPU's current stream."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_checks", nullptr, -1, functions, nullptr, nullptr, nullptr, nullptr};

// Whether Python and torch are those of the build (MOEDISP_BUILT_FOR: torch's
// version and commit).  If not, or if that cannot be told, ImportError is set.
bool as_built() {
    PyObject* hex = PySys_GetObject("hexversion");
    const unsigned long python = hex ? PyLong_AsUnsignedLong(hex) : 0;
    if (python >> 16 != (unsigned long)PY_VERSION_HEX >> 16) {
        PyErr_SetString(PyExc_ImportError, "_checks was built for another Python");
        return false;
    }
    THPObjectPtr version(PyImport_ImportModule("torch.version"));
    THPObjectPtr number(version ? PyObject_GetAttrString(version.get(), "__version__") : nullptr);
    THPObjectPtr commit(number ? PyObject_GetAttrString(version.get(), "git_version") : nullptr);
    THPObjectPtr both(commit ? PyUnicode_FromFormat("%S %S", number.get(), commit.get()) : nullptr);
    if (!both) {
        PyErr_SetString(PyExc_ImportError, "_checks was built for a torch that tells its version and commit");
        return false;
    }
    if (PyUnicode_CompareWithASCIIString(both.get(), MOEDISP_BUILT_FOR) != 0) {
        PyErr_Format(PyExc_ImportError, "_checks was built for torch %s, this is %S", MOEDISP_BUILT_FOR, both.get());
        return false;
    }
    return true;
}

}  // namespace

PyMODINIT_FUNC PyInit__checks() {
    if (!as_built()) return nullptr;
    type.tp_name = "combine_ep_get_dispatch_amd._checks.Checks";
    type.tp_basicsize = sizeof(Checks);
    type.tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_BASETYPE;
    type.tp_new = checks_new;
    type.tp_init = checks_init;
    type.tp_dealloc = checks_dealloc;
    type.tp_members = members;
    type.tp_methods = methods;
    if (PyType_Ready(&type) < 0) return nullptr;
    PyObject* m = PyModule_Create(&module);
    if (!m) return nullptr;
    Py_INCREF(&type);
    if (PyModule_AddObject(m, "Checks", reinterpret_cast<PyObject*>(&type)) < 0) return nullptr;
    return m;
}
