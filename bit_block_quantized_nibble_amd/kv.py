"""The paged key-value cache: binding of include/qbn_kv.h.

A decode step with 4-bit weights streams two things, the weights and the
key-value cache; this is the second. `KVCache` is the storage (bfloat16,
MXFP8 or MXFP4 pages), `KVPool` the bookkeeping (which pages each sequence
has), and the functions below write new tokens, attend over them and move
pages between steps, on torch's current stream and without the host reading
anything back. As in the rest of the package nothing is computed here: what the C ABI
cannot see (devices, dtypes, sizes) is checked, and pointers are passed.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import QbnError, _load, _need_dtype

KV_FORMATS = {"bf16": 16, "mxfp8": 7, "mxfp4": 1}
KV_EXPORTED = (
    "qbn_kv_struct_size", "qbn_kv_bytes", "qbn_kv_append", "qbn_kv_attention_workspace", "qbn_kv_attention_decode",
    "qbn_kv_attention_prefill", "qbn_kv_pool_workspace", "qbn_kv_reserve", "qbn_kv_fork", "qbn_kv_free",
    "qbn_kv_compact",
)
_I32 = torch.int32


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


_calls = None


def _call():
    """The module that makes the calls (csrc/kv_bind.cpp): checks, allocation,
    the C ABI. A launch takes 2.4 us of host time; ctypes took 3.4 to 5.9 more."""
    global _calls
    if _calls is None:
        _kv()
        try:
            from . import _kvcall
        except ImportError as e:
            raise RuntimeError("_kvcall.so is not built (%s); run `python -m bit_block_quantized_nibble_amd.build` "
                               "(or __graft_entry__.build()) first" % e)
        _calls = _kvcall
    return _calls


def _fixed(name: str, doc: str):
    """An attribute that stays the same tensor: the handle of a cache or pool
    holds its address. (`x.lens += 1` works in place and assigns the same one.)"""
    def put(self, t):
        if t is not getattr(self, "_" + name):
            raise AttributeError("%s is fixed for the life of the handle: write into it, or make another" % name)

    return property(lambda self: getattr(self, "_" + name), put, doc=doc)


def _first_device(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("the tensors of a cache or pool must be device (cuda) tensors")
    return t.get_device()


class KVCache:
    """Pages of keys and values in device memory (layouts: include/qbn_kv.h).

    k, v: [layers][pages][heads][page_size][head_dim] bfloat16 ("bf16"), uint8
    E4M3FN ("mxfp8"), or uint8 E2M1 pairs with a last axis of head_dim / 2
    ("mxfp4"); k_scales, v_scales: uint8 E8M0 [layers][pages][heads]
    [head_dim / 32][page_size] for the last two. The tensors are kept and used
    in place; they are fixed for the life of the handle."""

    k = _fixed("k", "Elements of K.")
    v = _fixed("v", "Elements of V.")
    k_scales = _fixed("k_scales", "E8M0 scales of K, or None.")
    v_scales = _fixed("v_scales", "E8M0 scales of V, or None.")

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
                raise ValueError("%s is on %s, the cache on another device" % (name, t.device))
        self.format, self._k, self._v, self._k_scales, self._v_scales = format, k, v, k_scales, v_scales
        self.layers, self.pages, self.heads, self.page_size, self.head_dim = layers, pages, heads, page, dim
        self.device, self.scale = k.device, 1.0 / math.sqrt(dim)
        self._handle = bytes(_CCache(
            KV_FORMATS[format], heads, dim, page, layers, pages, k.data_ptr(), v.data_ptr(),
            k_scales.data_ptr() if k_scales is not None else None, v_scales.data_ptr() if v_scales is not None else None))

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
    the page; 0 is free). The tensors are kept and used in place; they are fixed
    for the life of the handle (write into them, or make another pool)."""

    table = _fixed("table", "Pages of each slot, or -1.")
    lens = _fixed("lens", "Tokens of each slot.")
    refs = _fixed("refs", "How many entries name each page.")

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int):
        self._handle, self.index = (_calls or _call()).pool(table, lens, refs, page_size)
        self._table, self._lens, self._refs, self.page_size = table, lens, refs, page_size

    @classmethod
    def empty(cls, seqs: int, row: int, pages: int, page_size: int, device="cuda") -> "KVPool":
        """Slots without tokens, every page free."""
        return cls(torch.full((seqs, row), -1, dtype=torch.int32, device=device),
                   torch.zeros(seqs, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device), page_size)

    @classmethod
    def like(cls, other: "KVPool") -> "KVPool":
        """Uninitialized tables of the same sizes, as `out` of the calls below."""
        p = cls.__new__(cls)
        p._table, p._lens, p._refs, p._handle = (_calls or _call()).pool_like(other._table, other._lens, other._refs,
                                                                              other.page_size)
        p.page_size, p.index = other.page_size, other.index
        return p


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
              cu: Optional[torch.Tensor] = None, layer: int = 0) -> None:
    """Write new tokens' k, v ([tokens][heads][head_dim] float32 or bfloat16) into
    their pages. lens int32 [seqs] counts each sequence's tokens INCLUDING the
    new ones; cu int32 [seqs + 1] says which rows of k and v are whose (None: one
    new token per sequence). MX formats are quantized as quantize_mx does."""
    st = (_calls or _call()).append(cache._handle, cache.index, k, v, table, lens, cu, layer)
    if st:
        raise QbnError(st, "qbn_kv_append")


def _attention(decode: bool, cache, q, cu, table, lens, window, sinks, scale, layer, out, lse, workspace):
    got = (_calls or _call()).attention(decode, cache._handle, cache.index, q, cu, table, lens, window, sinks,
                                        cache.scale if scale is None else scale, layer, out, lse, workspace)
    if got.__class__ is int:
        raise QbnError(got, "qbn_kv_attention_decode" if decode else "qbn_kv_attention_prefill")
    return got


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
    with them is lens[b]; rows before cu[0] and from cu[seqs] on are padding
    (out = 0, lse = -inf). Otherwise as kv_attention_decode."""
    return _attention(False, cache, q, cu, table, lens, window, sinks, scale, layer, out, lse, workspace)


def _out(pool: KVPool, out: Optional[KVPool], cache: Optional[KVCache] = None) -> KVPool:
    out = pool if out is None else out
    if out.index != pool.index or (cache is not None and cache.index != pool.index):
        raise ValueError("the pools and the cache of a call must be on one device")
    return out


def _result(got, where: str) -> torch.Tensor:
    if got.__class__ is int:
        raise QbnError(got, where)
    return got


def kv_reserve(pool: KVPool, rows: torch.Tensor, tokens: torch.Tensor, out: Optional[KVPool] = None,
               status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Room for tokens[i] more tokens in slot rows[i] (int32 on the device): the
    slots grow, the lowest free pages are taken in the order of the requests.
    Returns a device int32: -1, or the first request that cannot be met (then
    nothing changes). `out`: other tables to write, in place without."""
    return _result((_calls or _call()).reserve(pool._handle, _out(pool, out)._handle, pool.index, rows, tokens, status,
                                               workspace), "qbn_kv_reserve")


def kv_fork(cache: KVCache, pool: KVPool, parents: torch.Tensor, children: torch.Tensor,
            out: Optional[KVPool] = None, status: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Slot children[i] (empty) becomes a copy of slot parents[i]: full pages are
    shared, a last page that is not full is copied in every layer. Returns the
    status word as kv_reserve does."""
    return _result((_calls or _call()).fork(cache._handle, pool._handle, _out(pool, out, cache)._handle, pool.index, parents,
                                            children, status, workspace), "qbn_kv_fork")


def kv_free(pool: KVPool, rows: torch.Tensor, window: int = 0, sinks: int = 0,
            out: Optional[KVPool] = None) -> None:
    """Give back the pages of slots rows[i]; with window > 0 only those that no
    later query of that window (and those sinks) sees, the slot going on."""
    st = (_calls or _call()).release(pool._handle, _out(pool, out)._handle, pool.index, rows, window, sinks)
    if st:
        raise QbnError(st, "qbn_kv_free")


def kv_compact(cache: KVCache, pool: KVPool, out: Optional[KVPool] = None, live: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Pack the pool: the L pages in use end up in pages 0 .. L - 1 of every
    layer, the tables follow. Returns L as a device int32."""
    return _result((_calls or _call()).compact(cache._handle, pool._handle, _out(pool, out, cache)._handle, pool.index,
                                               pool._table, live, workspace), "qbn_kv_compact")
