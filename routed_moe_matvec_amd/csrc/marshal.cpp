// The binding's part that every attention call goes through, compiled: a call of the
// smallest sizes takes the card 3 to 8 us, and reading its tensors' addresses, sizes and strides
// from Python and passing its arguments through ctypes took 3 to 5 longer than this (a step's norm and
// rotation 12.6 -> 8.2 us, one short decode 9.5 -> 6.1).
//
//  rows, array   the address of a tensor that is on the call's device, of its type and
//                large enough; for anything else what the binding's functions of the same
//                arguments, which look closer and say what is wrong, return or raise (otherwise(rows, array))
//  the calls     of qgemv.h by their own names, addresses and sizes as integers; every
//                call of the library runs without the interpreter's lock
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <tuple>
#include <type_traits>
#include <utility>

#include "qgemv.h"

namespace {

// A tensor of the library's own type (not a subclass, which may answer for itself) on that device.
const at::Tensor *plain_tensor(PyObject *o, long long device) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.defined() && t.is_cuda() && t.get_device() == device ? &t : nullptr;
}

bool numbers(PyObject *const *args, int n, long long *out) {
    for (int i = 0; i < n; ++i) {
        out[i] = PyLong_Check(args[i]) ? PyLong_AsLongLong(args[i]) : -1;
        if (out[i] < 0) {
            PyErr_Clear();
            return false;
        }
    }
    return true;
}

PyObject *other_rows, *other_array;

// rows(tensor, name, device, type, rows, width, ld): rows of `width` elements, `ld` elements apart
const void *find_rows(PyObject *const *args, Py_ssize_t n) {
    long long v[5];
    if (n != 7 || !numbers(args + 2, 5, v)) return nullptr;
    const long long type = v[1], count = v[2], width = v[3], ld = v[4];
    const at::Tensor *t = plain_tensor(args[0], v[0]);
    if (!t || t->dim() == 0 || count < 1 || count > INT_MAX || ld > INT_MAX) return nullptr;
    const at::ScalarType want = type == QG_TYPE_F32 ? at::kFloat : type == QG_TYPE_F16 ? at::kHalf : at::kBFloat16;
    if (type > QG_TYPE_BF16 || t->scalar_type() != want) return nullptr;
    const auto shape = t->sizes(), steps = t->strides();
    const long long have = t->numel();
    bool fits;
    if (t->is_contiguous() && (ld == width || have != shape[0] * width)) {  // folded in any way
        fits = (count - 1) * ld + width <= have;
    } else {
        fits = shape[0] >= count && (steps[0] == ld || shape[0] == 1);
        long long each = 1;
        for (int64_t i = t->dim() - 1; i > 0; --i) {
            fits = fits && (steps[i] == each || shape[i] == 1);
            each *= shape[i];
        }
        fits = fits && each == width;
    }
    return fits ? t->data_ptr() : nullptr;
}

// array(tensor, name, device, dtype, count): a dense tensor of `count` values of dtype, or of bytes (None)
const void *find_array(PyObject *const *args, Py_ssize_t n) {
    long long device, count;
    if (n != 5 || !numbers(args + 2, 1, &device) || !numbers(args + 4, 1, &count)) return nullptr;
    const at::Tensor *t = plain_tensor(args[0], device);
    if (!t || !t->is_contiguous()) return nullptr;
    long long have = t->numel();
    if (args[3] == Py_None)
        have *= t->element_size();
    else if (!THPDtype_Check(args[3]) || t->scalar_type() != reinterpret_cast<THPDtype *>(args[3])->scalar_type)
        return nullptr;
    return have < count ? nullptr : t->data_ptr();
}

// Tensors without memory of their own (those that vmap and grad wrap others in, sparse ones) throw where they
// are asked for it, or for strides: nothing may leave a C entry so, and the function of the same arguments says it.
template <auto FIND, PyObject **OTHER>
PyObject *address(PyObject *, PyObject *const *args, Py_ssize_t n) {
    const void *p = nullptr;
    try {
        p = FIND(args, n);
    } catch (const std::exception &) {
        PyErr_Clear();
    }
    if (p) return PyLong_FromVoidPtr(const_cast<void *>(p));
    return PyObject_Vectorcall(*OTHER, args, n, nullptr);
}

PyObject *otherwise(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 2) return PyErr_Format(PyExc_TypeError, "two functions are needed");
    Py_INCREF(args[0]);
    Py_INCREF(args[1]);
    Py_XSETREF(other_rows, args[0]);
    Py_XSETREF(other_array, args[1]);
    Py_RETURN_NONE;
}

template <class A>
A argument(PyObject *o) {
    if constexpr (std::is_pointer_v<A>) {
        return o == Py_None ? nullptr : static_cast<A>(PyLong_AsVoidPtr(o));
    } else if constexpr (std::is_same_v<A, float>) {
        return static_cast<float>(PyFloat_AsDouble(o));
    } else if constexpr (std::is_same_v<A, size_t>) {
        return PyLong_AsSize_t(o);
    } else {
        static_assert(std::is_same_v<A, int>);
        const long x = PyLong_AsLong(o);
        if (x > INT_MAX || x < INT_MIN) PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
        return static_cast<int>(x);
    }
}

template <class... A, size_t... I>
PyObject *invoke(int (*f)(A...), PyObject *const *args, Py_ssize_t n, std::index_sequence<I...>) {
    if (n != (Py_ssize_t)sizeof...(A)) {
        PyErr_Format(PyExc_TypeError, "%d arguments are needed, not %zd", (int)sizeof...(A), n);
        return nullptr;
    }
    std::tuple<A...> given{argument<A>(args[I])...};  // in order: an error stays set
    if (PyErr_Occurred()) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f(std::get<I>(given)...);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}
template <auto F, class... A>
PyObject *invoke_as(int (*f)(A...), PyObject *const *args, Py_ssize_t n) {
    return invoke(f, args, n, std::index_sequence_for<A...>());
}
template <auto F>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return invoke_as<F>(F, args, n);
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("rows", (address<find_rows, &other_rows>)),
                         METHOD("array", (address<find_array, &other_array>)),
                         METHOD("otherwise", otherwise),
                         METHOD("kv4_append", call<kv4_append>),
                         METHOD("kv4_gather", call<kv4_gather>),
                         METHOD("attn_decode_kv4", call<attn_decode_kv4>),
                         METHOD("attn_prefill", call<attn_prefill>),
                         METHOD("qk_norm_rope", call<qk_norm_rope>),
                         METHOD("attn_decode_kv4_sinks", call<attn_decode_kv4_sinks>),
                         METHOD("attn_prefill_sinks", call<attn_prefill_sinks>),
                         METHOD("attn_decode_kv4_prefix", call<attn_decode_kv4_prefix>),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
    other_rows = Py_NewRef(Py_None);
    other_array = Py_NewRef(Py_None);
    return PyModule_Create(&module);
}
