// Python entry points of the paged key-value cache's calls, and the module (_kvcall)
// of these and the other sources' calls.
//
// A decode step's cache calls are kernels of a few microseconds, and a launch
// takes 2.4 us of host time. Marshalling the arguments through ctypes took 3.4
// (append) to 5.9 us (attention) beside it, so these calls read the tensors
// here. Nothing else happens: it checks what the C ABI cannot
// see (devices, types, sizes) with the words of kv.py's other checks, allocates
// what the caller did not give, and returns the C ABI's status.
#include "kv_batch.h"

namespace {

using namespace qcall;

PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {  // cache, device, k, v, table, lens, cu, layer
    if (!count_is(n, 8)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *c = handle<qbn_kv_cache>(a[0]);
        const int64_t dev = integer(a[1]);
        const Rows k = vectors(tensor(a[2], "k"), c->heads, c->head_dim, dev, "k");
        const Rows v = vectors(tensor(a[3], "v"), c->heads, c->head_dim, dev, "v");
        const at::ScalarType t = k.t.scalar_type();
        if (t != at::kFloat && t != at::kBFloat16)
            refuse(PyExc_TypeError, "k dtype torch.%s (expected torch.float32, torch.bfloat16)", c10::toString(t));
        if (v.t.scalar_type() != t || v.t.size(0) != k.t.size(0)) refuse(PyExc_ValueError, "k and v must be alike");
        const qbn_kv_batch b = batch(dev, k.t.size(0), tensor(a[4], "table"), tensor(a[5], "lens"), a[6]);
        return PyLong_FromLong(qbn_kv_append(c, integer(a[7]), &b, k.t.data_ptr(), k.token, k.head, v.t.data_ptr(), v.token,
                                             v.head, t == at::kFloat ? QBN_F32 : QBN_BF16, OnDevice(dev)));
    });
}

// decode, cache, device, q, cu, table, lens, window, sinks, scale, layer, out, lse, workspace -> (out, lse), or a status
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 14)) return nullptr;
    return guarded([&]() -> PyObject * {
        const bool decode = a[0] == Py_True;
        const auto *c = handle<qbn_kv_cache>(a[1]);
        const int64_t dev = integer(a[2]);
        const Rows q = vectors(tensor(a[3], "q"), 0, c->head_dim, dev, "q");
        typed(q.t, at::kBFloat16, "torch.bfloat16", "q");
        const int64_t tokens = q.t.size(0), heads = q.t.size(1);
        const qbn_kv_batch b = batch(dev, tokens, tensor(a[5], "table"), tensor(a[6], "lens"), a[4]);
        const int32_t window = int32(a[7]), sinks = int32(a[8]);
        const double scale = PyFloat_AsDouble(a[9]);
        if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
        at::Tensor out, lse;
        if (a[11] == Py_None) {
            out = at::empty({tokens, heads, c->head_dim}, q.t.options());
        } else {
            out = tensor(a[11], "out");
            if (out.sizes() != q.t.sizes() || !out.is_contiguous())
                refuse(PyExc_ValueError, "out must be contiguous [tokens][heads][head_dim]");
            typed(out, at::kBFloat16, "torch.bfloat16", "out");
            if (index_of(out) != dev) elsewhere(out, "out");
        }
        if (a[12] == Py_None) {
            lse = at::empty({tokens, heads}, q.t.options().dtype(at::kFloat));
        } else {
            lse = tensor(a[12], "lse");
            if (lse.dim() != 2 || lse.size(0) != tokens || lse.size(1) != heads || !lse.is_contiguous())
                refuse(PyExc_ValueError, "lse must be contiguous [tokens][heads]");
            typed(lse, at::kFloat, "torch.float32", "lse");
            if (index_of(lse) != dev) elsewhere(lse, "lse");
        }
        const int64_t need = heads > INT32_MAX ? -1 : qbn_kv_attention_workspace(c, &b, (int32_t)heads, window, sinks, decode);
        const Workspace w = workspace(a[13], need, dev, q.t);
        const auto f = decode ? qbn_kv_attention_decode : qbn_kv_attention_prefill;
        const int32_t st = f(c, integer(a[10]), &b, heads > INT32_MAX ? -1 : (int32_t)heads, q.t.data_ptr(), q.token, q.head,
                             (float)scale, window, sinks, out.data_ptr(), (float *)lse.data_ptr(), w.p, w.bytes, OnDevice(dev));
        if (st) return PyLong_FromLong(st);
        PyObject *r = PyTuple_New(2);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(out)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(lse)));
        return r;
    });
}

PyObject *handle_of(const at::Tensor &table, const at::Tensor &lens, const at::Tensor &refs, int64_t page) {
    qbn_kv_pool p;
    p.seqs = table.size(0), p.row = table.size(1), p.pages = refs.numel();
    p.page_size = page > INT32_MAX || page < 0 ? -1 : (int32_t)page, p.reserved = 0;
    p.table = (int32_t *)table.data_ptr(), p.lens = (int32_t *)lens.data_ptr(), p.refs = (int32_t *)refs.data_ptr();
    return PyBytes_FromStringAndSize((const char *)&p, sizeof p);
}

PyObject *pool(PyObject *, PyObject *const *a, Py_ssize_t n) {  // table, lens, refs, page_size -> (handle, device)
    if (!count_is(n, 4)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &table = tensor(a[0], "table"), &lens = tensor(a[1], "lens"), &refs = tensor(a[2], "refs");
        typed(table, at::kInt, "torch.int32", "table");
        if (table.dim() != 2 || !table.is_contiguous())
            refuse(PyExc_ValueError, "table must be a contiguous [seqs][row] matrix");
        const int64_t dev = index_of(table);
        if (dev < 0) refuse(PyExc_ValueError, "the tensors of a cache or pool must be device (cuda) tensors");
        ints(lens, table.size(0), dev, "lens");
        ints(refs, refs.numel(), dev, "refs");
        return Py_BuildValue("NL", handle_of(table, lens, refs, integer(a[3])), (long long)dev);
    });
}

PyObject *pool_like(PyObject *, PyObject *const *a, Py_ssize_t n) {  // table, lens, refs, page_size -> (table, lens, refs, handle)
    if (!count_is(n, 4)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &table = tensor(a[0], "table"), &lens = tensor(a[1], "lens"), &refs = tensor(a[2], "refs");
        at::Tensor t = at::empty(table.sizes(), table.options()), l = at::empty(lens.sizes(), lens.options()),
                   r = at::empty(refs.sizes(), refs.options());
        PyObject *h = handle_of(t, l, r, integer(a[3]));
        return Py_BuildValue("NNNN", THPVariable_Wrap(std::move(t)), THPVariable_Wrap(std::move(l)),
                             THPVariable_Wrap(std::move(r)), h);
    });
}

// One device word: the caller's, or a new one.
at::Tensor word(PyObject *given, int64_t dev, const at::Tensor &like, const char *name) {
    if (given == Py_None) return at::empty({1}, like.options());
    const at::Tensor &t = tensor(given, name);
    ints(t, 1, dev, name);
    return t;
}

PyObject *status_and(int32_t st, at::Tensor &&t) {
    return st ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(t));
}

PyObject *reserve(PyObject *, PyObject *const *a, Py_ssize_t n) {  // in, out, device, rows, tokens, status, workspace
    if (!count_is(n, 7)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *in = handle<qbn_kv_pool>(a[0]), *out = handle<qbn_kv_pool>(a[1]);
        const int64_t dev = integer(a[2]);
        const at::Tensor &rows = tensor(a[3], "rows");
        const int64_t count = rows.numel();
        const int32_t *r = ints(rows, count, dev, "rows"), *t = ints(tensor(a[4], "tokens"), count, dev, "tokens");
        at::Tensor status = word(a[5], dev, rows, "status");
        const Workspace w = workspace(a[6], qbn_kv_pool_workspace(in, count), dev, rows);
        return status_and(qbn_kv_reserve(in, out, count, r, t, (int32_t *)status.data_ptr(), w.p, w.bytes, OnDevice(dev)),
                          std::move(status));
    });
}

PyObject *fork(PyObject *, PyObject *const *a, Py_ssize_t n) {  // cache, in, out, device, parents, children, status, workspace
    if (!count_is(n, 8)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *c = handle<qbn_kv_cache>(a[0]);
        const auto *in = handle<qbn_kv_pool>(a[1]), *out = handle<qbn_kv_pool>(a[2]);
        const int64_t dev = integer(a[3]);
        const at::Tensor &parents = tensor(a[4], "parents");
        const int64_t count = parents.numel();
        const int32_t *p = ints(parents, count, dev, "parents"), *k = ints(tensor(a[5], "children"), count, dev, "children");
        at::Tensor status = word(a[6], dev, parents, "status");
        const Workspace w = workspace(a[7], qbn_kv_pool_workspace(in, count), dev, parents);
        return status_and(qbn_kv_fork(c, in, out, count, p, k, (int32_t *)status.data_ptr(), w.p, w.bytes, OnDevice(dev)),
                          std::move(status));
    });
}

PyObject *release(PyObject *, PyObject *const *a, Py_ssize_t n) {  // in, out, device, rows, window, sinks
    if (!count_is(n, 6)) return nullptr;
    return guarded([&]() -> PyObject * {
        const int64_t dev = integer(a[2]);
        const at::Tensor &rows = tensor(a[3], "rows");
        return PyLong_FromLong(qbn_kv_free(handle<qbn_kv_pool>(a[0]), handle<qbn_kv_pool>(a[1]), rows.numel(),
                                           ints(rows, rows.numel(), dev, "rows"), int32(a[4]), int32(a[5]), OnDevice(dev)));
    });
}

PyObject *compact(PyObject *, PyObject *const *a, Py_ssize_t n) {  // cache, in, out, device, table, live, workspace
    if (!count_is(n, 7)) return nullptr;
    return guarded([&]() -> PyObject * {
        const auto *in = handle<qbn_kv_pool>(a[1]);
        const int64_t dev = integer(a[3]);
        const at::Tensor &like = tensor(a[4], "table");
        at::Tensor live = word(a[5], dev, like, "live");
        const Workspace w = workspace(a[6], qbn_kv_pool_workspace(in, 0), dev, like);
        return status_and(qbn_kv_compact(handle<qbn_kv_cache>(a[0]), in, handle<qbn_kv_pool>(a[2]), (int32_t *)live.data_ptr(),
                                         w.p, w.bytes, OnDevice(dev)),
                          std::move(live));
    });
}

#define QBN_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {QBN_METHOD(append),    QBN_METHOD(attention),   QBN_METHOD(pool),    QBN_METHOD(pool_like),
                           QBN_METHOD(reserve),   QBN_METHOD(fork),        QBN_METHOD(release), QBN_METHOD(compact),
                           QBN_METHOD(rope),      QBN_METHOD(append_rope), QBN_METHOD(moe_route),
                           QBN_METHOD(moe_experts), QBN_METHOD(moe),       {nullptr, nullptr, 0, nullptr}};
#undef QBN_METHOD

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kvcall", "Calls of the paged key-value cache, the rotation by positions and the experts' layer.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvcall() {
    PyObject *c = PyImport_ImportModule("torch._C");
    if (!c) return nullptr;
    g_raw_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
    g_exchange = PyObject_GetAttrString(c, "_cuda_exchangeDevice");
    g_exchange_back = PyObject_GetAttrString(c, "_cuda_maybeExchangeDevice");
    Py_DECREF(c);
    return g_raw_stream && g_exchange && g_exchange_back ? PyModule_Create(&g_module) : nullptr;
}
