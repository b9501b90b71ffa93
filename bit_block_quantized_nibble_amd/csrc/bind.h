// What the call module's entry points share (host code): reading tensors, checking
// what the C ABI cannot see, workspaces, streams and errors.
#pragma once

#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>

#include <string>

namespace qcall {

struct Refused {};  // a Python error is set

template <typename... A>
[[noreturn]] void refuse(PyObject *type, const char *form, A... a) {
    PyErr_Format(type, form, a...);
    throw Refused{};
}

inline std::string words(const at::Tensor &t) { return t.device().str(); }

inline const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

// `owner`: whose device the call runs on.
[[noreturn]] inline void elsewhere(const at::Tensor &t, const char *name, const char *owner = "the cache or pool") {
    refuse(PyExc_ValueError, "%s is on %s, %s on another device", name, words(t).c_str(), owner);
}

inline int64_t index_of(const at::Tensor &t) { return t.is_cuda() ? t.get_device() : -1; }

inline void typed(const at::Tensor &t, at::ScalarType want, const char *torch_name, const char *name) {
    if (t.scalar_type() != want)
        refuse(PyExc_TypeError, "%s dtype torch.%s (expected %s)", name, c10::toString(t.scalar_type()), torch_name);
}

// The address of an int32 vector of n entries on device dev.
inline int32_t *ints(const at::Tensor &t, int64_t n, int64_t dev, const char *name, const char *owner = "the cache or pool") {
    typed(t, at::kInt, "torch.int32", name);
    if (t.dim() != 1 || !t.is_contiguous()) refuse(PyExc_ValueError, "%s must be a contiguous vector", name);
    if (t.numel() != n) refuse(PyExc_ValueError, "%s has %lld entries; the call needs %lld", name, (long long)t.numel(), (long long)n);
    if (index_of(t) != dev) elsewhere(t, name, owner);
    return (int32_t *)t.data_ptr();
}

struct Rows {
    const at::Tensor &t;
    int64_t token, head;
};

// Strides of [tokens][heads][dim] vectors (views are taken as they are).
inline Rows vectors(const at::Tensor &t, int64_t heads, int64_t dim, int64_t dev, const char *name, const char *owner = "the cache or pool") {
    if (t.dim() != 3 || t.size(2) != dim || (heads && t.size(1) != heads))
        refuse(PyExc_ValueError, "%s must be [tokens][%s][%lld]", name, heads ? std::to_string(heads).c_str() : "heads", (long long)dim);
    if (t.stride(2) != 1) refuse(PyExc_ValueError, "the last axis of %s must be contiguous", name);
    if (index_of(t) != dev) elsewhere(t, name, owner);
    return {t, t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

// torch's current stream of a device, and the exchange of the current device for
// another (-1: none) and back, as torch's Python gives them.
inline PyObject *g_raw_stream = nullptr, *g_exchange = nullptr, *g_exchange_back = nullptr;

inline PyObject *with_index(PyObject *f, int64_t dev) {
    PyObject *arg = PyLong_FromLongLong(dev);
    PyObject *r = arg ? PyObject_CallOneArg(f, arg) : nullptr;
    Py_XDECREF(arg);
    return r;
}

// A call's stream, with its device as the current one while this lives: the
// default stream's handle is 0 on every device, and a launch on it goes to the
// current one.
class OnDevice {
  public:
    explicit OnDevice(int64_t dev) {
        PyObject *r = with_index(g_exchange, dev);
        if (!r) throw Refused{};
        before_ = PyLong_AsLongLong(r);
        Py_DECREF(r);
        moved_ = before_ >= 0 && before_ != dev;
        r = with_index(g_raw_stream, dev);
        if (r) {
            stream_ = PyLong_AsVoidPtr(r);
            Py_DECREF(r);
        }
        if (!stream_ && PyErr_Occurred()) {
            back();
            throw Refused{};
        }
    }
    OnDevice(const OnDevice &) = delete;
    ~OnDevice() { back(); }
    operator void *() const { return stream_; }

  private:
    void back() {
        if (!moved_) return;
        moved_ = false;
        PyObject *type, *value, *trace;  // an error on its way is kept
        PyErr_Fetch(&type, &value, &trace);
        PyObject *r = with_index(g_exchange_back, before_);
        if (r) Py_DECREF(r);
        else PyErr_WriteUnraisable(g_exchange_back);
        PyErr_Restore(type, value, trace);
    }
    int64_t before_ = -1;
    bool moved_ = false;
    void *stream_ = nullptr;
};

inline int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
// The C ABI refuses what does not fit its 32-bit arguments' ranges; the value must not wrap into them first.
inline int32_t int32(PyObject *o) {
    const int64_t v = integer(o);
    return v > INT32_MAX || v < INT32_MIN ? INT32_MIN : (int32_t)v;
}

// A handle: the bytes of its C struct, made by kv.py.
template <typename T>
const T *handle(PyObject *o) {
    if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != sizeof(T)) refuse(PyExc_TypeError, "not a handle of this library");
    return reinterpret_cast<const T *>(PyBytes_AS_STRING(o));
}

// The workspace of a call: the caller's, or one of `need` bytes.
struct Workspace {
    at::Tensor keep;
    void *p = nullptr;
    int64_t bytes = 0;
};
inline Workspace workspace(PyObject *given, int64_t need, int64_t dev, const at::Tensor &like, const char *owner = "the cache or pool") {
    Workspace w;
    if (given != Py_None) {
        const at::Tensor &t = tensor(given, "workspace");
        const int64_t have = t.numel() * t.element_size();
        if (have < need)
            refuse(PyExc_ValueError, "workspace holds %lld bytes; the call needs %lld", (long long)have, (long long)need);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
        if (index_of(t) != dev) elsewhere(t, "workspace", owner);
        w.p = t.data_ptr(), w.bytes = have;
    } else if (need > 0) {
        w.keep = at::empty({need}, like.options().dtype(at::kByte));
        w.p = w.keep.data_ptr(), w.bytes = need;
    }
    return w;
}

template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const Refused &) {
    } catch (...) {  // torch's, the allocator's torch.OutOfMemoryError above all: as torch's own functions raise it
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

inline bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
    return false;
}

// Entry points of the other sources, for the module's table.
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *moe_route(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *moe_experts(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *moe(PyObject *, PyObject *const *a, Py_ssize_t n);

}  // namespace qcall
