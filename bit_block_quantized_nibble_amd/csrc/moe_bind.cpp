// Python entry points of the experts' layer (part of the module _kvcall): what
// kv_bind.cpp does for the cache's calls.
#include "../../include/qbn_moe.h"
#include "bind.h"

namespace qcall {
namespace {

constexpr const char *kOwner = "the layer";

// x or out: bfloat16 [tokens][hidden], rows anywhere.
int64_t stride_of(const at::Tensor &t, int64_t hidden, int64_t dev, const char *name) {
    typed(t, at::kBFloat16, "torch.bfloat16", name);
    if (t.dim() != 2 || t.size(1) != hidden) refuse(PyExc_ValueError, "%s must be [tokens][%lld]", name, (long long)hidden);
    if (t.stride(1) != 1) refuse(PyExc_ValueError, "the last axis of %s must be contiguous", name);
    if (index_of(t) != dev) elsewhere(t, name, kOwner);
    return t.size(0) > 1 ? t.stride(0) : hidden;
}

// ids or weights: contiguous [tokens][top_k], the caller's or new ones.
at::Tensor choice(PyObject *given, int64_t tokens, int64_t top, at::ScalarType type, const char *torch_name, int64_t dev,
                  const at::Tensor &like, const char *name) {
    if (given == Py_None) return at::empty({tokens, top}, like.options().dtype(type));
    const at::Tensor &t = tensor(given, name);
    typed(t, type, torch_name, name);
    if (t.dim() != 2 || t.size(0) != tokens || (top >= 0 && t.size(1) != top) || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous [tokens][top_k]", name);
    if (index_of(t) != dev) elsewhere(t, name, kOwner);
    return t;
}

at::Tensor output(PyObject *given, const at::Tensor &x, int64_t dev, int64_t *stride) {
    at::Tensor out = given == Py_None ? at::empty(x.sizes(), x.options()) : tensor(given, "out");
    if (out.dim() != 2 || out.size(0) != x.size(0)) refuse(PyExc_ValueError, "out must be [tokens][hidden] as x");
    *stride = stride_of(out, x.size(1), dev, "out");
    return out;
}

PyObject *tuple_of(at::Tensor *t, int n) {
    PyObject *r = PyTuple_New(n);
    if (!r) return nullptr;
    for (int i = 0; i < n; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(t[i])));
    return r;
}

}  // namespace

// router, device, x, ids, weights, workspace -> (ids, weights), or a status
PyObject *moe_route(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 6)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *r = handle<qbn_moe_router>(a[0]);
        const int64_t dev = integer(a[1]);
        const at::Tensor &x = tensor(a[2], "x");
        const int64_t xs = stride_of(x, r->hidden, dev, "x"), tokens = x.size(0);
        at::Tensor t[2] = {choice(a[3], tokens, r->top_k, at::kInt, "torch.int32", dev, x, "ids"),
                           choice(a[4], tokens, r->top_k, at::kFloat, "torch.float32", dev, x, "weights")};
        const Workspace w = workspace(a[5], qbn_moe_workspace(r, nullptr, tokens, r->top_k), dev, x, kOwner);
        const int32_t st = qbn_moe_route(r, tokens, x.data_ptr(), xs, (int32_t *)t[0].data_ptr(), (float *)t[1].data_ptr(),
                                         w.p, w.bytes, OnDevice(dev));
        return st ? PyLong_FromLong(st) : tuple_of(t, 2);
    });
}

// experts, device, x, ids, weights, out, workspace -> out, or a status
PyObject *moe_experts(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 7)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *e = handle<qbn_moe_weights>(a[0]);
        const int64_t dev = integer(a[1]);
        const at::Tensor &x = tensor(a[2], "x");
        const int64_t xs = stride_of(x, e->hidden, dev, "x"), tokens = x.size(0);
        if (a[3] == Py_None || a[4] == Py_None) refuse(PyExc_TypeError, "ids and weights must be tensors");
        const at::Tensor ids = choice(a[3], tokens, -1, at::kInt, "torch.int32", dev, x, "ids");
        const at::Tensor weights = choice(a[4], tokens, ids.size(1), at::kFloat, "torch.float32", dev, x, "weights");
        const int32_t top = ids.size(1) > INT32_MAX ? -1 : (int32_t)ids.size(1);
        int64_t os;
        at::Tensor out = output(a[5], x, dev, &os);
        const Workspace w = workspace(a[6], qbn_moe_workspace(nullptr, e, tokens, top), dev, x, kOwner);
        const int32_t st = qbn_moe_experts(e, tokens, top, x.data_ptr(), xs, (const int32_t *)ids.data_ptr(),
                                           (const float *)weights.data_ptr(), out.data_ptr(), os, w.p, w.bytes, OnDevice(dev));
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(out));
    });
}

// router, experts, device, x, out, ids, weights, workspace -> (out, ids, weights), or a status
PyObject *moe(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 8)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *r = handle<qbn_moe_router>(a[0]);
        const auto *e = handle<qbn_moe_weights>(a[1]);
        const int64_t dev = integer(a[2]);
        const at::Tensor &x = tensor(a[3], "x");
        const int64_t xs = stride_of(x, r->hidden, dev, "x"), tokens = x.size(0);
        int64_t os;
        at::Tensor t[3];
        t[0] = output(a[4], x, dev, &os);
        t[1] = choice(a[5], tokens, r->top_k, at::kInt, "torch.int32", dev, x, "ids");
        t[2] = choice(a[6], tokens, r->top_k, at::kFloat, "torch.float32", dev, x, "weights");
        const Workspace w = workspace(a[7], qbn_moe_workspace(r, e, tokens, r->top_k), dev, x, kOwner);
        const int32_t st = qbn_moe(r, e, tokens, x.data_ptr(), xs, (int32_t *)t[1].data_ptr(), (float *)t[2].data_ptr(),
                                   t[0].data_ptr(), os, w.p, w.bytes, OnDevice(dev));
        return st ? PyLong_FromLong(st) : tuple_of(t, 3);
    });
}

}  // namespace qcall
