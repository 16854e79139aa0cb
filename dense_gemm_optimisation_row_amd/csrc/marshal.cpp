// Calls of forms seen before, for the layers whose kernels take about as long as
// a call's host time (layers.py): finds the form by its arguments' shapes, strides,
// types and devices, allocates the outputs and the workspace and calls the C entry
// point.  A form is made, checked and kept by layers.py; what is not known here is
// left to it.  Nothing of a tensor is kept, neither its address nor its identity.
//
// In Python a call of six tensors takes 8.0 us, so 4.5, of which the launch is 2.6.
#define PY_SSIZE_T_CLEAN
#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <pybind11/gil.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <memory>
#include <unordered_map>
#include <utility>
#include <vector>

namespace {

constexpr size_t kMostForms = 4096;   // then they are dropped
constexpr int kMostPointers = 12;

struct Key {
    int64_t v[192];
    int n = 0;
    bool full = false;
    void add(int64_t x)
    {
        if (n < 192)
            v[n++] = x;
        else
            full = true;
    }
    uint64_t hash() const
    {
        uint64_t h = 0x9e3779b97f4a7c15ull;
        for (int i = 0; i < n; ++i) {
            h ^= (uint64_t)v[i];
            h *= 0xff51afd7ed558ccdull;
            h ^= h >> 32;
        }
        return h;
    }
};

struct Output {
    int given;   // which of the tensors it is, or -1
    std::vector<int64_t> sizes;
    at::ScalarType type;
};
struct Form {
    std::vector<int64_t> key;
    std::vector<char> params;
    std::vector<int> slots;   // of the pointer arguments: a tensor, or -1 - an output
    std::vector<Output> outputs;
    uintptr_t entry;
    int64_t workspace;        // bytes; -1: the entry point takes none
};
std::unordered_multimap<uint64_t, std::shared_ptr<Form>> forms;   // under the interpreter's lock

// The key of a call; false where it is not one for here: another kind of tensor,
// or one that requires grad where torch records gradients (layers.py refuses it).
bool make_key(Key &k, PyObject *op, PyObject *tensors, PyObject *extra, const at::Tensor *const (&found)[16], int64_t device)
{
    k.add(PyLong_AsLongLong(op));
    const Py_ssize_t count = PyTuple_GET_SIZE(tensors), more = PyTuple_GET_SIZE(extra);
    const bool grad = at::GradMode::is_enabled();
    for (Py_ssize_t i = 0; i < more; ++i)
        k.add(PyLong_AsLongLong(PyTuple_GET_ITEM(extra, i)));
    for (Py_ssize_t i = 0; i < count; ++i) {
        const at::Tensor *t = found[i];
        if (!t) {
            k.add(-1);
            continue;
        }
        if (!t->is_cuda() || t->layout() != c10::kStrided || (grad && t->requires_grad()) ||
            t->device().index() != device)
            return false;
        k.add((int64_t)t->scalar_type() | (int64_t)t->dim() << 8 |
              (t->scalar_type() == at::kChar && ((uintptr_t)t->data_ptr() & 15) ? 1 << 16 : 0));
        for (const int64_t s : t->sizes())
            k.add(s);
        for (const int64_t s : t->strides())
            k.add(s);
    }
    return !k.full && !PyErr_Occurred();
}

// The tensors themselves, which the caller's tuple holds.
bool unpack(PyObject *tensors, PyObject *extra, const at::Tensor *(&found)[16])
{
    if (!PyTuple_Check(tensors) || !PyTuple_Check(extra) || PyTuple_GET_SIZE(tensors) > 16) {
        PyErr_SetString(PyExc_TypeError, "tensors and extra are tuples, of at most 16 tensors");
        return false;
    }
    const Py_ssize_t n = PyTuple_GET_SIZE(tensors);
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject *o = PyTuple_GET_ITEM(tensors, i);
        found[i] = nullptr;
        if (o == Py_None)
            continue;
        if (!THPVariable_Check(o)) {
            PyErr_SetString(PyExc_TypeError, "expected a tensor or None");
            return false;
        }
        found[i] = &THPVariable_Unpack(o);
    }
    return true;
}

std::shared_ptr<Form> find(const Key &k)
{
    const auto range = forms.equal_range(k.hash());
    for (auto it = range.first; it != range.second; ++it)
        if ((int)it->second->key.size() == k.n && memcmp(it->second->key.data(), k.v, sizeof(int64_t) * k.n) == 0)
            return it->second;
    return nullptr;
}

template <size_t... I>
int call_with(uintptr_t entry, const uintptr_t *a, std::index_sequence<I...>)
{
    return ((int (*)(decltype((void)I, (uintptr_t)0)...))entry)(a[I]...);
}
int call(uintptr_t entry, const uintptr_t *a, int n)   // integers and pointers only
{
    switch (n) {
    case 5: return call_with(entry, a, std::make_index_sequence<5>());
    case 11: return call_with(entry, a, std::make_index_sequence<11>());
    default: return -1;
    }
}

// keep(op, tensors, extra, device, entry, params, slots, outputs, workspace):
// outputs are indices of given tensors or (sizes, dtype).
PyObject *keep(PyObject *, PyObject *args)
{
    HANDLE_TH_ERRORS
    PyObject *op, *tensors, *extra, *slots, *outputs;
    long long device, entry, workspace;
    const char *params;
    Py_ssize_t bytes;
    if (!PyArg_ParseTuple(args, "OOOLLy#OOL", &op, &tensors, &extra, &device, &entry, &params, &bytes, &slots, &outputs,
                          &workspace))
        return nullptr;
    const at::Tensor *found[16];
    if (!unpack(tensors, extra, found))
        return nullptr;
    Key k;
    auto f = std::make_shared<Form>();
    const Py_ssize_t n = PyTuple_Size(slots), outs = PyTuple_Size(outputs);
    const int total = 1 + (int)n + (workspace >= 0 ? 2 : 0) + 1;
    if (n < 0 || outs < 0 || (total != 5 && total != 11)) {
        PyErr_SetString(PyExc_ValueError, "no such entry point");
        return nullptr;
    }
    if (!make_key(k, op, tensors, extra, found, device)) {
        if (PyErr_Occurred())
            return nullptr;
        Py_RETURN_NONE;
    }
    for (Py_ssize_t i = 0; i < n; ++i)
        f->slots.push_back((int)PyLong_AsLong(PyTuple_GET_ITEM(slots, i)));
    for (Py_ssize_t i = 0; i < outs; ++i) {
        PyObject *o = PyTuple_GET_ITEM(outputs, i);
        Output out{-1, {}, at::kByte};
        if (PyLong_Check(o)) {
            out.given = (int)PyLong_AsLong(o);
        } else {
            PyObject *sizes = PyTuple_GetItem(o, 0), *type = PyTuple_GetItem(o, 1);
            if (!sizes || !type || !THPDtype_Check(type)) {
                PyErr_SetString(PyExc_TypeError, "an output is an index or (sizes, dtype)");
                return nullptr;
            }
            for (Py_ssize_t d = 0; d < PyTuple_Size(sizes); ++d)
                out.sizes.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(sizes, d)));
            out.type = reinterpret_cast<THPDtype *>(type)->scalar_type;
        }
        f->outputs.push_back(std::move(out));
    }
    for (const int s : f->slots)
        if (s >= (int)PyTuple_GET_SIZE(tensors) || -1 - s >= (int)outs) {
            PyErr_SetString(PyExc_ValueError, "no such tensor or output");
            return nullptr;
        }
    if (PyErr_Occurred())
        return nullptr;
    f->key.assign(k.v, k.v + k.n);
    f->params.assign(params, params + bytes);
    f->entry = (uintptr_t)entry;
    f->workspace = workspace;
    if (forms.size() >= kMostForms)
        forms.clear();
    if (!find(k))
        forms.emplace(k.hash(), std::move(f));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// run(op, tensors, extra, device, stream): the outputs, a status other than 0, or
// None where the form is not known.
PyObject *run(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    HANDLE_TH_ERRORS
    if (nargs != 5) {
        PyErr_SetString(PyExc_TypeError, "run takes 5 arguments");
        return nullptr;
    }
    const at::Tensor *found[16];
    if (!unpack(args[1], args[2], found))
        return nullptr;
    const int64_t device = PyLong_AsLongLong(args[3]);
    Key k;
    if (!make_key(k, args[0], args[1], args[2], found, device)) {
        if (PyErr_Occurred())
            return nullptr;
        Py_RETURN_NONE;
    }
    const std::shared_ptr<Form> f = find(k);   // held, should another thread drop the forms
    if (!f)
        Py_RETURN_NONE;
    const uintptr_t stream = (uintptr_t)PyLong_AsUnsignedLongLong(args[4]);
    if (PyErr_Occurred())
        return nullptr;
    const auto options = at::TensorOptions().device(at::Device(at::kCUDA, (c10::DeviceIndex)device));
    at::Tensor made[4], space;
    const at::Tensor *out[4];
    const int outs = (int)f->outputs.size();
    if (outs > 4 || f->slots.size() > (size_t)kMostPointers) {
        PyErr_SetString(PyExc_ValueError, "too many outputs");
        return nullptr;
    }
    int rc;
    {
        // without the lock, as torch's and ctypes' calls: an allocation or a launch may
        // wait for the GPU, and that for another thread.  The caller holds the tensors.
        pybind11::gil_scoped_release unlocked;
        for (int i = 0; i < outs; ++i) {
            const Output &o = f->outputs[i];
            if (o.given < 0)
                made[i] = at::empty(o.sizes, options.dtype(o.type));
            out[i] = o.given < 0 ? &made[i] : found[o.given];
        }
        uintptr_t a[kMostPointers + 4];
        int n = 0;
        a[n++] = (uintptr_t)f->params.data();
        for (const int s : f->slots) {
            const at::Tensor *t = s >= 0 ? found[s] : out[-1 - s];
            a[n++] = t ? (uintptr_t)t->data_ptr() : 0;
        }
        if (f->workspace >= 0) {
            if (f->workspace > 0)
                space = at::empty({f->workspace}, options.dtype(at::kByte));
            a[n++] = f->workspace > 0 ? (uintptr_t)space.data_ptr() : 0;
            a[n++] = (uintptr_t)f->workspace;
        }
        a[n++] = stream;
        rc = call(f->entry, a, n);
    }
    if (rc != 0)
        return PyLong_FromLong(rc);
    if (outs == 1)
        return THPVariable_Wrap(*out[0]);
    PyObject *t = PyTuple_New(outs);
    for (int i = 0; t && i < outs; ++i)
        PyTuple_SET_ITEM(t, i, THPVariable_Wrap(*out[i]));
    return t;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {{"keep", keep, METH_VARARGS, nullptr},
                         {"run", (PyCFunction)(void (*)(void))run, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
