// Python entry points of the rotation by positions (part of the module _kvcall): what
// kv_bind.cpp does for the cache's calls.
#include "../../include/qbn_rope.h"
#include "kv_batch.h"

namespace qcall {
namespace {

constexpr const char *kOwner = "the rotation";

int32_t dtype_of(const at::Tensor &t, const char *name) {
    const at::ScalarType s = t.scalar_type();
    if (s != at::kFloat && s != at::kBFloat16)
        refuse(PyExc_TypeError, "%s dtype torch.%s (expected torch.float32, torch.bfloat16)", name, c10::toString(s));
    return s == at::kFloat ? QBN_F32 : QBN_BF16;
}

// [tokens][heads][dim] vectors to write: the caller's (any strides, the last axis contiguous) or new ones.
at::Tensor vectors_out(PyObject *given, const at::Tensor &like, at::ScalarType type, const char *torch_name, int64_t dev, const char *owner) {
    if (given == Py_None) return at::empty(like.sizes(), like.options().dtype(type));
    const at::Tensor &t = tensor(given, "out");
    if (t.sizes() != like.sizes()) refuse(PyExc_ValueError, "out must be [tokens][heads][dim] as its source");
    typed(t, type, torch_name, "out");
    vectors(t, 0, like.size(2), dev, "out", owner);
    return t;
}

}  // namespace

PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {  // rotation, device, x, positions, out -> out, or a status
    if (!count_is(n, 5)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *r = handle<qbn_rotation>(a[0]);
        const int64_t dev = integer(a[1]);
        const at::Tensor &t = tensor(a[2], "x");
        if (t.dim() != 3) refuse(PyExc_ValueError, "x must be [tokens][heads][dim]");
        const int64_t tokens = t.size(0), heads = t.size(1), dim = t.size(2);
        const Rows x = vectors(t, 0, dim, dev, "x", kOwner);
        const int32_t dtype = dtype_of(t, "x");
        const int32_t *pos = ints(tensor(a[3], "positions"), tokens, dev, "positions", kOwner);
        at::Tensor out = vectors_out(a[4], t, t.scalar_type(), dtype == QBN_F32 ? "torch.float32" : "torch.bfloat16", dev, kOwner);
        const Rows o = vectors(out, 0, dim, dev, "out", kOwner);
        // A rotation made on the host is on the same "device" as host tensors: their addresses are no kernel's.
        if (dev < 0) refuse(PyExc_ValueError, "x and the rotation must be on a device (cuda); x is on %s", words(t).c_str());
        const auto small = [](int64_t v) { return v > INT32_MAX ? -1 : (int32_t)v; };  // refused, not wrapped
        const int32_t st = qbn_rope(r, tokens, small(heads), small(dim), pos, t.data_ptr(), x.token, x.head, out.data_ptr(),
                                    o.token, o.head, dtype, OnDevice(dev));
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(out));
    });
}

// cache, device, q, k, v, table, lens, cu, layer, rotation, its device, out -> out (None without q), or a status
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 12)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *c = handle<qbn_kv_cache>(a[0]);
        const int64_t dev = integer(a[1]);
        const Rows k = vectors(tensor(a[3], "k"), c->heads, c->head_dim, dev, "k");
        const Rows v = vectors(tensor(a[4], "v"), c->heads, c->head_dim, dev, "v");
        const int32_t dtype = dtype_of(k.t, "k");
        if (v.t.scalar_type() != k.t.scalar_type() || v.t.size(0) != k.t.size(0)) refuse(PyExc_ValueError, "k and v must be alike");
        const auto *r = handle<qbn_rotation>(a[9]);
        if (integer(a[10]) != dev) refuse(PyExc_ValueError, "the rotation is on another device than the cache");
        const int64_t tokens = k.t.size(0);
        at::Tensor out;
        const void *q = nullptr;
        void *to = nullptr;
        int64_t heads = 0, qt = 0, qh = 0, ot = 0, oh = 0;
        if (a[2] == Py_None) {
            if (a[11] != Py_None) refuse(PyExc_ValueError, "out is for q, which is None");
        } else {
            const Rows rows = vectors(tensor(a[2], "q"), 0, c->head_dim, dev, "q");
            if (rows.t.scalar_type() != k.t.scalar_type() || rows.t.size(0) != tokens) refuse(PyExc_ValueError, "q and k must be alike");
            heads = rows.t.size(1), q = rows.t.data_ptr(), qt = rows.token, qh = rows.head;
            out = vectors_out(a[11], rows.t, at::kBFloat16, "torch.bfloat16", dev, "the cache or pool");
            const Rows o = vectors(out, 0, c->head_dim, dev, "out");
            to = out.data_ptr(), ot = o.token, oh = o.head;
        }
        const qbn_kv_batch b = batch(dev, tokens, tensor(a[5], "table"), tensor(a[6], "lens"), a[7]);
        const int32_t st = qbn_kv_append_rope(c, integer(a[8]), &b, r, heads > INT32_MAX ? -1 : (int32_t)heads, q, qt, qh, to, ot, oh,
                                              k.t.data_ptr(), k.token, k.head, v.t.data_ptr(), v.token, v.head, dtype, OnDevice(dev));
        if (st) return PyLong_FromLong(st);
        if (a[2] == Py_None) Py_RETURN_NONE;
        return THPVariable_Wrap(std::move(out));
    });
}

}  // namespace qcall
