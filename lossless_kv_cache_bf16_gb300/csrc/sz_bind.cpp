// sz_bind.cpp -- the part of the Python binding that every call of a serving
// operator goes through, in C++: checks of tensor arguments, and the calls of
// the C ABI.  Interpreted, they cost more time than a decode step's kernels.
//
// It sees tensors only through their Python attributes (dtype, shape,
// stride(), is_cuda, get_device(), is_contiguous(), data_ptr()), and the library only
// through the addresses that splitzip.py passes, so that it depends on neither
// PyTorch's headers nor the order in which libraries are loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <cstring>

#include "splitzip.h"
#include "sz_rows.h"

namespace {

PyObject *s_dtype, *s_shape, *s_stride, *s_is_cuda, *s_is_contiguous, *s_data_ptr, *s_numel, *s_get_device;

// An owned reference.
struct Ref {
    PyObject* o;
    explicit Ref(PyObject* p = nullptr) : o(p) {}
    ~Ref() { Py_XDECREF(o); }
    Ref(const Ref&) = delete;
    Ref& operator=(const Ref&) = delete;
    explicit operator bool() const { return o != nullptr; }
};

// 1 or 0 for a truth value (its reference is taken over), -1 with an error.
int truth(PyObject* o) {
    if (!o) return -1;
    const int r = PyObject_IsTrue(o);
    Py_DECREF(o);
    return r;
}

PyObject* refuse(PyObject* what, const char* why) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%U %s", what, why);
    return nullptr;
}

// extra: how many further arguments may follow
bool expect(Py_ssize_t got, Py_ssize_t want, Py_ssize_t extra = 0) {
    if (got >= want && got <= want + extra) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, not %zd", want, got);
    return false;
}

// Whether t is on the GPU of that number (on any one if it is negative): the
// kernels run on the call's GPU, and a pointer into another would be followed
// there.  False with an error.
bool on_gpu(PyObject* t, long device, PyObject* what) {
    if (device >= 0) {
        Ref index(PyObject_CallMethodNoArgs(t, s_get_device));
        if (!index) return false;
        const long got = PyLong_AsLong(index.o);
        if (got == device) return true;
        if (got == -1 && PyErr_Occurred()) return false;
    }
    const int cuda = truth(PyObject_GetAttr(t, s_is_cuda));
    if (cuda < 0) return false;
    if (!cuda) return refuse(what, "must be a CUDA tensor");
    if (device >= 0) return refuse(what, "must be on the GPU that the call runs on");
    return true;
}
// The device argument after the first n, -1 without one; -2 with an error.
long device_of(PyObject* const* a, Py_ssize_t n, Py_ssize_t got) {
    if (got <= n) return -1;
    const long d = PyLong_AsLong(a[n]);
    return d == -1 && PyErr_Occurred() ? -2 : d;
}

// (data_ptr, shape, stride) of a bf16 CUDA tensor [rows, heads, channels] whose
// channels are contiguous.
PyObject* rows_of(PyObject* t, PyObject* bfloat16, PyObject* what, long device) {
    if (device < -1) return nullptr;
    Ref dtype(PyObject_GetAttr(t, s_dtype)), shape(PyObject_GetAttr(t, s_shape)), stride(PyObject_CallMethodNoArgs(t, s_stride));
    if (!dtype || !shape || !stride) return nullptr;
    if (dtype.o != bfloat16 || !PyTuple_Check(shape.o) || !PyTuple_Check(stride.o) || PyTuple_GET_SIZE(shape.o) != 3 ||
        PyTuple_GET_SIZE(stride.o) != 3)
        return refuse(what, "must be a bfloat16 tensor of three dimensions");
    if (!on_gpu(t, device, what)) return nullptr;
    const long long last = PyLong_AsLongLong(PyTuple_GET_ITEM(stride.o, 2));
    if (last != 1) {
        if (PyErr_Occurred()) return nullptr;
        bool empty = false;
        for (int k = 0; k < 3; k++) empty |= PyLong_AsLongLong(PyTuple_GET_ITEM(shape.o, k)) == 0;
        if (PyErr_Occurred()) return nullptr;
        if (!empty) return refuse(what, "must have contiguous channels");
    }
    Ref ptr(PyObject_CallMethodNoArgs(t, s_data_ptr));
    if (!ptr) return nullptr;
    return PyTuple_Pack(3, ptr.o, shape.o, stride.o);
}

// The checks below take the number of the GPU that the call runs on as a last
// argument; without it (or with -1) any will do.

// rows(t, bfloat16, what[, device])
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return expect(n, 3, 1) ? rows_of(a[0], a[1], a[2], device_of(a, 3, n)) : nullptr;
}

// written_rows(t, bfloat16, shape, what[, device]): the same for a tensor of that shape
// which a kernel writes: no two of its rows may share memory.
PyObject* written_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 4, 1)) return nullptr;
    PyObject* what = a[3];
    Ref got(rows_of(a[0], a[1], what, device_of(a, 4, n)));
    if (!got) return nullptr;
    PyObject *shape = PyTuple_GET_ITEM(got.o, 1), *stride = PyTuple_GET_ITEM(got.o, 2);
    const int same = PyObject_RichCompareBool(shape, a[2], Py_EQ);
    if (same < 0) return nullptr;
    if (!same) {
        PyErr_Format(PyExc_ValueError, "%U must have shape %R, not %R", what, a[2], shape);
        return nullptr;
    }
    // From the smallest stride on, each must reach past all that lies below.
    long long size[3], step[3];
    for (int k = 0; k < 3; k++) {
        size[k] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, k));
        step[k] = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, k));
    }
    if (PyErr_Occurred()) return nullptr;
    bool done[3] = {};
    long long reach = 0;
    const bool empty = size[0] == 0 || size[1] == 0 || size[2] == 0;
    for (int turn = 0; turn < 3 && !empty; turn++) {
        int next = -1;
        for (int k = 0; k < 3; k++)
            if (!done[k] && (next < 0 || step[k] < step[next])) next = k;
        done[next] = true;
        if (size[next] <= 1) continue;
        if (step[next] <= reach) return refuse(what, "must not overlap itself");
        reach += step[next] * (size[next] - 1);
    }
    Py_INCREF(got.o);
    return got.o;
}

// overlap(a, b): whether two results of rows() or written_rows() share memory.
PyObject* overlap(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 2)) return nullptr;
    sz::RowSet set[2];
    uint64_t dim = 0;
    for (int k = 0; k < 2; k++) {
        PyObject *ptr, *shape, *stride;
        unsigned long long size[3];
        long long step[3];
        if (!PyArg_ParseTuple(a[k], "OO!O!", &ptr, &PyTuple_Type, &shape, &PyTuple_Type, &stride) ||
            !PyArg_ParseTuple(shape, "KKK", &size[0], &size[1], &size[2]) ||
            !PyArg_ParseTuple(stride, "LLL", &step[0], &step[1], &step[2]))
            return nullptr;
        set[k] = {PyLong_AsVoidPtr(ptr), step[0], step[1], size[0], size[1]};
        if (PyErr_Occurred()) return nullptr;
        dim = k == 0 || size[2] > dim ? size[2] : dim;
    }
    return PyBool_FromLong(sz::rows_overlap(set[0], set[1], dim));
}

// Whether t has the values of a tensor of that shape, in its own shape if it
// has as many dimensions.  False with an error.
bool holds(PyObject* t, PyObject* want, PyObject* what) {
    Ref shape(PyObject_GetAttr(t, s_shape));
    if (!shape) return false;
    if (PyTuple_Check(shape.o) && PyTuple_GET_SIZE(shape.o) == PyTuple_GET_SIZE(want)) {
        const int same = PyObject_RichCompareBool(shape.o, want, Py_EQ);
        if (same == 0) PyErr_Format(PyExc_ValueError, "%U must have shape %R, not %R", what, want, shape.o);
        return same > 0;
    }
    long long values = 1;
    for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(want); k++) values *= PyLong_AsLongLong(PyTuple_GET_ITEM(want, k));
    Ref numel(PyObject_CallMethodNoArgs(t, s_numel));
    if (!numel || PyErr_Occurred()) return false;
    const long long got = PyLong_AsLongLong(numel.o);
    if (got != values && !PyErr_Occurred())
        PyErr_Format(PyExc_ValueError, "%U must hold %lld values, not %lld", what, values, got);
    return got == values;
}

// pointer(t, dtype or None, count, what[, device]) -> data_ptr of a contiguous
// CUDA tensor of that type; None for None.  count: its number of values, its
// shape (a flat tensor, or one of other dimensions, need only hold as many
// values), or -1.
PyObject* pointer(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 4, 1)) return nullptr;
    PyObject *t = a[0], *what = a[3];
    if (t == Py_None) Py_RETURN_NONE;
    const long device = device_of(a, 4, n);
    if (device < -1) return nullptr;
    if (a[1] != Py_None) {
        Ref dtype(PyObject_GetAttr(t, s_dtype));
        if (!dtype) return nullptr;
        if (dtype.o != a[1]) {
            PyErr_Format(PyExc_ValueError, "%U must be %S", what, a[1]);
            return nullptr;
        }
    }
    if (PyTuple_Check(a[2])) {
        if (!holds(t, a[2], what)) return nullptr;
    }
    const long long want = PyTuple_Check(a[2]) ? -1 : PyLong_AsLongLong(a[2]);
    if (want == -1 && PyErr_Occurred()) return nullptr;
    if (want >= 0) {
        Ref numel(PyObject_CallMethodNoArgs(t, s_numel));
        if (!numel) return nullptr;
        const long long got = PyLong_AsLongLong(numel.o);
        if (got == -1 && PyErr_Occurred()) return nullptr;
        if (got != want) {
            PyErr_Format(PyExc_ValueError, "%U must hold %lld values, not %lld", what, want, got);
            return nullptr;
        }
    }
    if (!on_gpu(t, device, what)) return nullptr;
    const int dense = truth(PyObject_CallMethodNoArgs(t, s_is_contiguous));
    if (dense < 0) return nullptr;
    if (!dense) return refuse(what, "must be contiguous");
    return PyObject_CallMethodNoArgs(t, s_data_ptr);
}

// ---- calls: the function's address, then its arguments ----------------------
// Pointers are integers or None, the stream the last one.  Bad Python values
// leave an error that is looked at once, before the call.
void* as_ptr(PyObject* o) { return o == Py_None ? nullptr : PyLong_AsVoidPtr(o); }
int64_t as_int(PyObject* o) { return PyLong_AsLongLong(o); }
size_t as_size(PyObject* o) { return PyLong_AsSize_t(o); }
float as_float(PyObject* o) { return (float)PyFloat_AsDouble(o); }

template <typename F>
F* address(PyObject* o) {
    return reinterpret_cast<F*>(PyLong_AsVoidPtr(o));
}

#define P(k) as_ptr(a[k])
#define I(k) as_int(a[k])
#define Z(k) as_size(a[k])

// Evaluates the arguments, then calls, unless one of them was bad.
template <typename F, typename... Args>
PyObject* invoke(F* f, Args... args) {
    if (PyErr_Occurred()) return nullptr;
    if (!f) {
        PyErr_SetString(PyExc_ValueError, "no function");
        return nullptr;
    }
    // Other threads run while a full launch queue holds the call up.
    PyThreadState* state = PyEval_SaveThread();
    const long status = (long)f(args...);
    PyEval_RestoreThread(state);
    return PyLong_FromLong(status);
}

template <typename T>
T* to(void* p) {
    return static_cast<T*>(p);
}

PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 25)) return nullptr;
    return invoke(address<decltype(sz_qk_norm_rope)>(a[0]), P(1), I(2), I(3), Z(4), P(5), I(6), I(7), Z(8), Z(9), Z(10), P(11),
                  P(12), as_float(a[13]), to<const float>(P(14)), Z(15), (int)I(16), to<const int32_t>(P(17)), P(18), I(19),
                  I(20), P(21), I(22), I(23), to<CUstream_st>(P(24)));
}

PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 19)) return nullptr;
    return invoke(address<decltype(sz_cache_append)>(a[0]), P(1), I(2), I(3), P(4), I(5), I(6), Z(7), to<const int64_t>(P(8)),
                  to<const int32_t>(P(9)), P(10), Z(11), Z(12), Z(13), Z(14), to<float>(P(15)), to<int32_t>(P(16)),
                  to<int>(P(17)), to<CUstream_st>(P(18)));
}

PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 16)) return nullptr;
    return invoke(address<decltype(sz_cache_read)>(a[0]), P(1), Z(2), Z(3), Z(4), Z(5), to<const int64_t>(P(6)), Z(7), P(8),
                  I(9), I(10), P(11), I(12), I(13), to<int>(P(14)), to<CUstream_st>(P(15)));
}

PyObject* cache_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 24)) return nullptr;
    return invoke(address<decltype(sz_cache_attend)>(a[0]), P(1), I(2), I(3), Z(4), Z(5), P(6), Z(7), Z(8), Z(9), Z(10),
                  to<const int32_t>(P(11)), Z(12), to<const int32_t>(P(13)), as_float(a[14]), P(15), I(16), I(17),
                  to<float>(P(18)), to<float>(P(19)), to<int>(P(20)), P(21), Z(22), to<CUstream_st>(P(23)));
}

PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 20)) return nullptr;
    return invoke(address<decltype(sz_cache_evict)>(a[0]), P(1), Z(2), Z(3), Z(4), Z(5), to<const int32_t>(P(6)), Z(7),
                  to<const int32_t>(P(8)), to<const int32_t>(P(9)), Z(10), Z(11), Z(12), to<float>(P(13)), to<int32_t>(P(14)),
                  to<int32_t>(P(15)), to<int>(P(16)), P(17), Z(18), to<CUstream_st>(P(19)));
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rows),        FAST(written_rows), FAST(overlap),      FAST(pointer),      FAST(qk_norm_rope), FAST(cache_append),
                         FAST(cache_read),  FAST(cache_attend), FAST(cache_evict),  {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sz_bind", "Checks and calls of splitzip.py's serving operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sz_bind(void) {
    struct {
        PyObject** at;
        const char* name;
    } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"}, {&s_is_cuda, "is_cuda"},
                 {&s_is_contiguous, "is_contiguous"}, {&s_data_ptr, "data_ptr"}, {&s_numel, "numel"},
                 {&s_get_device, "get_device"}};
    for (auto& x : names)
        if (!(*x.at = PyUnicode_InternFromString(x.name))) return nullptr;
    return PyModule_Create(&module);
}
