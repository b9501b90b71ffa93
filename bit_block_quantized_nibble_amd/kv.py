"""The paged key-value cache: binding of include/qbn_kv.h.

A decode step with 4-bit weights streams two things, the weights and the
key-value cache; this is the second. `KVCache` is the storage (bfloat16,
MXFP8 or MXFP4 pages), `KVPool` the bookkeeping (which pages each sequence
has), and the functions below write new tokens, attend over them and move
pages between steps, on torch's current stream and without the host reading
anything back. As in the rest of the package this module only marshals: it
checks what the C ABI cannot see (devices, dtypes, sizes) and passes pointers.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import QbnError, _load, _need, _need_dtype

KV_FORMATS = {"bf16": 16, "mxfp8": 7, "mxfp4": 1}
KV_EXPORTED = (
    "qbn_kv_struct_size", "qbn_kv_bytes", "qbn_kv_append", "qbn_kv_attention_workspace", "qbn_kv_attention_decode",
    "qbn_kv_attention_prefill", "qbn_kv_pool_workspace", "qbn_kv_reserve", "qbn_kv_fork", "qbn_kv_free",
    "qbn_kv_compact",
)
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_I32, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32
# torch's current stream of a device as an integer: what
# torch.cuda.current_stream(device).cuda_stream gives, without making a Stream
# object (1.9 us of a small call's 14).
_raw_stream = torch._C._cuda_getCurrentRawStream


class _CCache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("layers", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p)]


class _CBatch(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int64), ("tokens", ctypes.c_int64), ("row", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("cu", ctypes.c_void_p)]


class _CPool(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int64), ("row", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p)]


_bound = None


def _kv():
    """libqbn with the argument types of its cache entry points."""
    global _bound
    if _bound is not None:
        return _bound
    lib = _load()
    P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    C, B, L = ctypes.POINTER(_CCache), ctypes.POINTER(_CBatch), ctypes.POINTER(_CPool)
    lib.qbn_kv_struct_size.argtypes, lib.qbn_kv_struct_size.restype = [I32], ctypes.c_size_t
    for name, args, res in (
            ("qbn_kv_bytes", [I32, I64, I64, I32, I32, I32, I32], I64),
            ("qbn_kv_append", [C, I64, B, P, I64, I64, P, I64, I64, I32, P], I32),
            ("qbn_kv_attention_workspace", [C, B, I32, I32, I32, I32], I64),
            ("qbn_kv_attention_decode", [C, I64, B, I32, P, I64, I64, F32, I32, I32, P, P, P, I64, P], I32),
            ("qbn_kv_attention_prefill", [C, I64, B, I32, P, I64, I64, F32, I32, I32, P, P, P, I64, P], I32),
            ("qbn_kv_pool_workspace", [L, I64], I64),
            ("qbn_kv_reserve", [L, L, I64, P, P, P, P, I64, P], I32),
            ("qbn_kv_fork", [C, L, L, I64, P, P, P, P, I64, P], I32),
            ("qbn_kv_free", [L, L, I64, P, I32, I32, P], I32),
            ("qbn_kv_compact", [C, L, L, P, P, I64, P], I32)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res
    for which, struct in enumerate((_CCache, _CBatch, _CPool)):
        if lib.qbn_kv_struct_size(which) != ctypes.sizeof(struct):
            raise RuntimeError("libqbn ABI mismatch: rebuild the library")
    _bound = lib
    return lib


def kv_nbytes(format: str, layers: int, pages: int, heads: int, page_size: int, head_dim: int, part: int = 0) -> int:
    """Bytes of K's (equally V's) elements (part 0) or scales (part 1); -1 if invalid."""
    return int(_kv().qbn_kv_bytes(KV_FORMATS[format], layers, pages, heads, page_size, head_dim, part))


# The checks below run before every call, next to kernels of a few
# microseconds: they compare device indexes and types without building
# objects, and leave the words to the branch that raises.

def _elsewhere(t: torch.Tensor, name: str):
    raise ValueError("%s is on %s, the cache or pool on another device" % (name, t.device))


def _first_device(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("the tensors of a cache or pool must be device (cuda) tensors")
    return t.get_device()


def _ints(t: torch.Tensor, n: int, dev: int, name: str) -> int:
    """The address of an int32 vector of n entries on device dev."""
    if t.dtype is not _I32:
        _need_dtype(t, (_I32,), name)
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector" % name)
    if t.numel() != n:
        raise ValueError("%s has %d entries; the call needs %d" % (name, t.numel(), n))
    if t.get_device() != dev:
        _elsewhere(t, name)
    return t.data_ptr()


class KVCache:
    """Pages of keys and values in device memory (layouts: include/qbn_kv.h).

    k, v: [layers][pages][heads][page_size][head_dim] bfloat16 ("bf16"), uint8
    E4M3FN ("mxfp8"), or uint8 E2M1 pairs with a last axis of head_dim / 2
    ("mxfp4"); k_scales, v_scales: uint8 E8M0 [layers][pages][heads]
    [head_dim / 32][page_size] for the last two. The tensors are kept and used
    in place; they are fixed for the life of the handle."""

    def __init__(self, format: str, k: torch.Tensor, v: torch.Tensor, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None):
        if format not in KV_FORMATS:
            raise ValueError("unknown cache format %r" % (format,))
        dt = torch.bfloat16 if format == "bf16" else torch.uint8
        if k.dim() != 5 or k.shape != v.shape:
            raise ValueError("k and v must be [layers][pages][heads][page_size][head_dim], alike")
        layers, pages, heads, page, dim = k.shape
        dim *= 2 if format == "mxfp4" else 1
        need = kv_nbytes(format, layers, pages, heads, page, dim)
        if need < 0:
            raise ValueError("unsupported cache shape: layers, pages and heads at least 1, page_size 16 to 256 (a power "
                             "of two), head_dim 64, 96, 128, 192 or 256; got %s" % (tuple(k.shape),))
        parts = [(k, "k"), (v, "v")]
        if format == "bf16":
            if k_scales is not None or v_scales is not None:
                raise ValueError("a bf16 cache has no scales")
        else:
            for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
                if t is None or tuple(t.shape) != (layers, pages, heads, dim // 32, page):
                    raise ValueError("%s must be [layers][pages][heads][head_dim / 32][page_size]" % name)
                parts.append((t, name))
        for t, name in parts:
            _need_dtype(t, (dt if name in ("k", "v") else torch.uint8,), name)
            if not t.is_contiguous():
                raise ValueError("%s must be contiguous" % name)
        self.index = _first_device(k)
        for t, name in parts:
            if t.get_device() != self.index:
                _elsewhere(t, name)
        self.format, self.k, self.v, self.k_scales, self.v_scales = format, k, v, k_scales, v_scales
        self.layers, self.pages, self.heads, self.page_size, self.head_dim = layers, pages, heads, page, dim
        self.device, self.scale = k.device, 1.0 / math.sqrt(dim)
        self._c = _CCache(KV_FORMATS[format], heads, dim, page, layers, pages, k.data_ptr(), v.data_ptr(),
                          k_scales.data_ptr() if k_scales is not None else None,
                          v_scales.data_ptr() if v_scales is not None else None)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, format: str, layers: int, pages: int, heads: int, page_size: int, head_dim: int,
              device="cuda") -> "KVCache":
        """A cache with uninitialized pages (attention reads only tokens that were appended)."""
        if format not in KV_FORMATS:
            raise ValueError("unknown cache format %r" % (format,))
        shape = (layers, pages, heads, page_size, head_dim // 2 if format == "mxfp4" else head_dim)
        dt = torch.bfloat16 if format == "bf16" else torch.uint8
        k, v = torch.empty(shape, dtype=dt, device=device), torch.empty(shape, dtype=dt, device=device)
        if format == "bf16":
            return cls(format, k, v)
        s = (layers, pages, heads, head_dim // 32, page_size)
        return cls(format, k, v, torch.empty(s, dtype=torch.uint8, device=device),
                   torch.empty(s, dtype=torch.uint8, device=device))


class KVPool:
    """Which pages each sequence slot has: table int32 [seqs][row] (a page or
    -1), lens int32 [seqs] (tokens), refs int32 [pages] (how many entries name
    the page; 0 is free)."""

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int):
        _need_dtype(table, (_I32,), "table")
        if table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be a contiguous [seqs][row] matrix")
        self.index = _first_device(table)
        seqs, row = table.shape
        self.table, self.lens, self.refs, self.page_size = table, lens, refs, int(page_size)
        pages = refs.numel()
        self._c = _CPool(seqs, row, pages, self.page_size, 0, table.data_ptr(), _ints(lens, seqs, self.index, "lens"),
                         _ints(refs, pages, self.index, "refs"))
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, seqs: int, row: int, pages: int, page_size: int, device="cuda") -> "KVPool":
        """Slots without tokens, every page free."""
        return cls(torch.full((seqs, row), -1, dtype=torch.int32, device=device),
                   torch.zeros(seqs, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device), page_size)

    @classmethod
    def like(cls, other: "KVPool") -> "KVPool":
        """Uninitialized tables of the same sizes, as `out` of the calls below."""
        return cls(torch.empty_like(other.table), torch.empty_like(other.lens), torch.empty_like(other.refs),
                   other.page_size)


def _batch(dev: int, tokens: int, table: torch.Tensor, lens: torch.Tensor, cu: Optional[torch.Tensor]) -> _CBatch:
    if table.dtype is not _I32:
        _need_dtype(table, (_I32,), "table")
    if table.dim() != 2:
        raise ValueError("table must be [seqs][row] with contiguous rows")
    seqs, row = table.shape
    if table.is_contiguous():
        stride = row
    else:
        if row > 1 and table.stride(1) != 1:
            raise ValueError("table must be [seqs][row] with contiguous rows")
        stride = table.stride(0) if seqs > 1 else row
    if table.get_device() != dev:
        _elsewhere(table, "table")
    if cu is None:
        if tokens != seqs:
            raise ValueError("%d tokens for %d sequences: one each is wanted without cu" % (tokens, seqs))
        return _CBatch(seqs, tokens, row, stride, table.data_ptr(), _ints(lens, seqs, dev, "lens"), None)
    return _CBatch(seqs, tokens, row, stride, table.data_ptr(), _ints(lens, seqs, dev, "lens"),
                   _ints(cu, seqs + 1, dev, "cu"))


def _vectors(t: torch.Tensor, heads: int, dim: int, dev: int, name: str):
    """Strides of [tokens][heads][dim] vectors (views are taken as they are)."""
    if t.dim() != 3 or t.shape[2] != dim or (heads and t.shape[1] != heads):
        raise ValueError("%s must be [tokens][%s][%d], got %s" % (name, heads or "heads", dim, tuple(t.shape)))
    a, b, c = t.stride()
    if c != 1:
        raise ValueError("the last axis of %s must be contiguous" % name)
    if t.get_device() != dev:
        _elsewhere(t, name)
    return a if t.shape[0] > 1 else 0, b if t.shape[1] > 1 else 0


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
              cu: Optional[torch.Tensor] = None, layer: int = 0) -> None:
    """Write new tokens' k, v ([tokens][heads][head_dim] float32 or bfloat16) into
    their pages. lens int32 [seqs] counts each sequence's tokens INCLUDING the
    new ones; cu int32 [seqs + 1] says which rows of k and v are whose (None: one
    new token per sequence). MX formats are quantized as quantize_mx does."""
    lib, dev = _bound or _kv(), cache.index
    kt, kh = _vectors(k, cache.heads, cache.head_dim, dev, "k")
    vt, vh = _vectors(v, cache.heads, cache.head_dim, dev, "v")
    dtype, tokens = _DTYPES.get(k.dtype), k.shape[0]
    if dtype is None:
        _need_dtype(k, (torch.float32, torch.bfloat16), "k")
    if v.dtype is not k.dtype or v.shape[0] != tokens:
        raise ValueError("k and v must be alike")
    b = _batch(dev, tokens, table, lens, cu)
    st = lib.qbn_kv_append(cache._ref, layer, b, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, dtype, _raw_stream(dev))
    if st:
        raise QbnError(st, "qbn_kv_append")


def _attention(decode: bool, cache, q, cu, table, lens, window, sinks, scale, layer, out, lse, workspace):
    lib, dev, dim = _bound or _kv(), cache.index, cache.head_dim
    qt, qh = _vectors(q, 0, dim, dev, "q")
    if q.dtype is not _BF16:
        _need_dtype(q, (_BF16,), "q")
    tokens, heads, _ = shape = q.shape
    b = _batch(dev, tokens, table, lens, cu)
    if out is None:
        out = q.new_empty(shape)
    else:
        if out.shape != shape or not out.is_contiguous():
            raise ValueError("out must be contiguous [tokens][heads][head_dim]")
        _need_dtype(out, (_BF16,), "out")
        if out.get_device() != dev:
            _elsewhere(out, "out")
    if lse is None:
        lse = q.new_empty((tokens, heads), dtype=_F32)
    else:
        if lse.shape != shape[:2] or not lse.is_contiguous():
            raise ValueError("lse must be contiguous [tokens][heads]")
        _need_dtype(lse, (_F32,), "lse")
        if lse.get_device() != dev:
            _elsewhere(lse, "lse")
    need = lib.qbn_kv_attention_workspace(cache._ref, b, heads, window, sinks, decode)
    ws = None
    if workspace is not None:
        ws, need = _given_workspace(workspace, need, dev)
    elif need > 0:
        workspace = q.new_empty(need, dtype=torch.uint8)
        ws = workspace.data_ptr()
    fn = lib.qbn_kv_attention_decode if decode else lib.qbn_kv_attention_prefill
    st = fn(cache._ref, layer, b, heads, q.data_ptr(), qt, qh, cache.scale if scale is None else scale, window, sinks,
            out.data_ptr(), lse.data_ptr(), ws, need, _raw_stream(dev))
    if st:
        raise QbnError(st, "qbn_kv_attention_decode" if decode else "qbn_kv_attention_prefill")
    return out, lse


def _given_workspace(t: torch.Tensor, need: int, dev: int):
    _need(t, need, "workspace")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if t.get_device() != dev:
        _elsewhere(t, "workspace")
    return t.data_ptr(), t.numel() * t.element_size()


def kv_attention_decode(cache: KVCache, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, window: int = 0,
                        sinks: int = 0, scale: Optional[float] = None, layer: int = 0,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """Attention of one new token per sequence (q bfloat16 [seqs][q_heads]
    [head_dim], at position lens - 1) over the cache: (out bfloat16 [seqs]
    [q_heads][head_dim], lse float32 [seqs][q_heads], natural log). window > 0
    keeps the last `window` tokens and the first `sinks` visible; scale defaults
    to 1 / sqrt(head_dim)."""
    return _attention(True, cache, q, None, table, lens, window, sinks, scale, layer, out, lse, workspace)


def kv_attention_prefill(cache: KVCache, q: torch.Tensor, cu: Optional[torch.Tensor], table: torch.Tensor,
                         lens: torch.Tensor, window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                         layer: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None):
    """Causal attention of chunks of new tokens (already appended): rows
    cu[b] .. cu[b + 1] - 1 of q are the last tokens of sequence b, whose length
    with them is lens[b]. Otherwise as kv_attention_decode."""
    return _attention(False, cache, q, cu, table, lens, window, sinks, scale, layer, out, lse, workspace)


def _out(pool: KVPool, out: Optional[KVPool], cache: Optional[KVCache] = None) -> KVPool:
    out = pool if out is None else out
    if out.index != pool.index:
        _elsewhere(out.table, "out")
    if cache is not None and cache.index != pool.index:
        _elsewhere(pool.table, "pool")
    return out


def _pool_workspace(lib, pool: KVPool, count: int, workspace: Optional[torch.Tensor]):
    """(the tensor, its address, its bytes)"""
    need = lib.qbn_kv_pool_workspace(pool._ref, count)
    if workspace is None:
        workspace = pool.table.new_empty(max(need, 0) // 4)
        return workspace, workspace.data_ptr(), need
    return (workspace,) + _given_workspace(workspace, need, pool.index)


def _word(t: Optional[torch.Tensor], pool: KVPool, name: str) -> torch.Tensor:
    if t is None:
        return pool.table.new_empty(1)
    _ints(t, 1, pool.index, name)
    return t


def kv_reserve(pool: KVPool, rows: torch.Tensor, tokens: torch.Tensor, out: Optional[KVPool] = None,
               status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Room for tokens[i] more tokens in slot rows[i] (int32 on the device): the
    slots grow, the lowest free pages are taken in the order of the requests.
    Returns a device int32: -1, or the first request that cannot be met (then
    nothing changes). `out`: other tables to write, in place without."""
    lib, out, dev, n = _bound or _kv(), _out(pool, out), pool.index, rows.numel()
    r, t = _ints(rows, n, dev, "rows"), _ints(tokens, n, dev, "tokens")
    status = _word(status, pool, "status")
    workspace, ws, size = _pool_workspace(lib, pool, n, workspace)
    st = lib.qbn_kv_reserve(pool._ref, out._ref, n, r, t, status.data_ptr(), ws, size, _raw_stream(dev))
    if st:
        raise QbnError(st, "qbn_kv_reserve")
    return status


def kv_fork(cache: KVCache, pool: KVPool, parents: torch.Tensor, children: torch.Tensor,
            out: Optional[KVPool] = None, status: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Slot children[i] (empty) becomes a copy of slot parents[i]: full pages are
    shared, a last page that is not full is copied in every layer. Returns the
    status word as kv_reserve does."""
    lib, out, dev, n = _bound or _kv(), _out(pool, out, cache), pool.index, parents.numel()
    a, c = _ints(parents, n, dev, "parents"), _ints(children, n, dev, "children")
    status = _word(status, pool, "status")
    workspace, ws, size = _pool_workspace(lib, pool, n, workspace)
    st = lib.qbn_kv_fork(cache._ref, pool._ref, out._ref, n, a, c, status.data_ptr(), ws, size, _raw_stream(dev))
    if st:
        raise QbnError(st, "qbn_kv_fork")
    return status


def kv_free(pool: KVPool, rows: torch.Tensor, window: int = 0, sinks: int = 0,
            out: Optional[KVPool] = None) -> None:
    """Give back the pages of slots rows[i]; with window > 0 only those that no
    later query of that window (and those sinks) sees, the slot going on."""
    lib, out, dev, n = _bound or _kv(), _out(pool, out), pool.index, rows.numel()
    st = lib.qbn_kv_free(pool._ref, out._ref, n, _ints(rows, n, dev, "rows"), window, sinks, _raw_stream(dev))
    if st:
        raise QbnError(st, "qbn_kv_free")


def kv_compact(cache: KVCache, pool: KVPool, out: Optional[KVPool] = None, live: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Pack the pool: the L pages in use end up in pages 0 .. L - 1 of every
    layer, the tables follow. Returns L as a device int32."""
    lib, out = _bound or _kv(), _out(pool, out, cache)
    live = _word(live, pool, "live")
    workspace, ws, size = _pool_workspace(lib, pool, 0, workspace)
    st = lib.qbn_kv_compact(cache._ref, pool._ref, out._ref, live.data_ptr(), ws, size, _raw_stream(pool.index))
    if st:
        raise QbnError(st, "qbn_kv_compact")
    return live
