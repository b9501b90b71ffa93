"""The mixture-of-experts layer over 4-bit weights: binding of include/qbn_moe.h.

`MoERouter` chooses the experts of a token, `MoE` has their weights; `moe_route`
is the choice, `moe_experts` the experts' products, `moe` both in one call. As in
the rest of the package nothing is computed here: what the C ABI cannot see
(devices, dtypes, sizes) is checked, and pointers are passed.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import QbnError, _load, _need_dtype, kv
from .kv import _fixed

MOE_FORMATS = {"mxfp4": 1, "nvfp4": 2}
MOE_EXPORTED = ("qbn_moe_struct_size", "qbn_moe_workspace", "qbn_moe_route", "qbn_moe_experts", "qbn_moe")


class _CRouter(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("normalize", ctypes.c_int32), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class _CWeights(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("experts", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("w13", ctypes.c_void_p), ("w13_scales", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_scales", ctypes.c_void_p), ("w13_scale2", ctypes.c_void_p),
                ("w2_scale2", ctypes.c_void_p)]


_bound = None


def _moe_lib():
    """libqbn with the argument types of the layer's entry points."""
    global _bound
    if _bound is not None:
        return _bound
    lib = _load()
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    R, W = ctypes.POINTER(_CRouter), ctypes.POINTER(_CWeights)
    lib.qbn_moe_struct_size.argtypes, lib.qbn_moe_struct_size.restype = [I32], ctypes.c_size_t
    for name, args, res in (
            ("qbn_moe_workspace", [R, W, I64, I32], I64),
            ("qbn_moe_route", [R, I64, P, I64, P, P, P, I64, P], I32),
            ("qbn_moe_experts", [W, I64, I32, P, I64, P, P, P, I64, P, I64, P], I32),
            ("qbn_moe", [R, W, I64, P, I64, P, P, P, I64, P, I64, P], I32)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res
    for which, struct in enumerate((_CRouter, _CWeights)):
        if lib.qbn_moe_struct_size(which) != ctypes.sizeof(struct):
            raise RuntimeError("libqbn ABI mismatch: rebuild the library")
    _bound = lib
    return lib


def _part(t, shape, dtype, name, index=None):
    """A part of a layer: its sizes, dtype, memory and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    _need_dtype(t, (dtype,), name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s; got %s" % (name, list(shape), list(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device (cuda) tensor" % name)
    if index is not None and t.get_device() != index:
        raise ValueError("%s is on %s, the layer on another device" % (name, t.device))
    return t.data_ptr()


class MoERouter:
    """weight: bfloat16 [experts][hidden]; bias: float32 [experts] or None. The
    top_k experts of the largest logits are a token's; their weights are the
    softmax over these (normalize) or over all logits."""

    weight = _fixed("weight", "[experts][hidden].")
    bias = _fixed("bias", "[experts], or None.")

    def __init__(self, weight: torch.Tensor, top_k: int, bias: Optional[torch.Tensor] = None, normalize: bool = True):
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
            raise ValueError("weight must be a tensor [experts][hidden]")
        experts, hidden = weight.shape
        if not 1 <= experts <= 1024 or not 1 <= top_k <= min(experts, 32) or hidden % 32 or not 32 <= hidden <= 1 << 16:
            raise ValueError("unsupported router: 1 to 1024 experts, top_k 1 to 32 of them, hidden a multiple of 32 up "
                             "to 65536; got %d experts, top_k %d, hidden %d" % (experts, top_k, hidden))
        p = _part(weight, (experts, hidden), torch.bfloat16, "weight")
        self.index = weight.get_device()
        b = None if bias is None else _part(bias, (experts,), torch.float32, "bias", self.index)
        self._weight, self._bias, self.top_k, self.normalize = weight, bias, int(top_k), bool(normalize)
        self.experts, self.hidden = experts, hidden
        _moe_lib()
        self._handle = bytes(_CRouter(experts, self.top_k, hidden, int(self.normalize), p, b))


class MoE:
    """Experts' weights in "mxfp4" or "nvfp4", and the router that chooses among
    them (None: moe_experts only). w13: uint8 E2M1 pairs [experts][2 inter]
    [hidden / 2], the gate's rows before the up projection's; w2 [experts][hidden]
    [inter / 2]; scales uint8 with hidden / 32 and inter / 32 columns (nvfp4: / 16);
    nvfp4 also takes a float32 factor per expert of each (any finite ones). The
    tensors are kept and used in place; they are fixed for the life of the
    handle."""

    w13 = _fixed("w13", "Codes of gate and up projection.")
    w13_scales = _fixed("w13_scales", "Their scales.")
    w2 = _fixed("w2", "Codes of the down projection.")
    w2_scales = _fixed("w2_scales", "Its scales.")
    w13_scale2 = _fixed("w13_scale2", "[experts] (nvfp4), or None.")
    w2_scale2 = _fixed("w2_scale2", "[experts] (nvfp4), or None.")
    router = _fixed("router", "The MoERouter, or None.")

    def __init__(self, format: str, router: Optional[MoERouter], w13: torch.Tensor, w13_scales: torch.Tensor,
                 w2: torch.Tensor, w2_scales: torch.Tensor, w13_scale2: Optional[torch.Tensor] = None,
                 w2_scale2: Optional[torch.Tensor] = None):
        if format not in MOE_FORMATS:
            raise ValueError("unknown or unsupported format %r (expected mxfp4 or nvfp4)" % (format,))
        for t, name in ((w13, "w13"), (w2, "w2")):
            if not isinstance(t, torch.Tensor) or t.dim() != 3:
                raise ValueError("%s must be a tensor [experts][rows][k / 2]" % name)
        experts, hidden, inter = w13.shape[0], w2.shape[1], w2.shape[2] * 2
        if not 1 <= experts <= 1024 or hidden % 32 or inter % 32 or not 32 <= hidden <= 1 << 16 or not 32 <= inter <= 1 << 16:
            raise ValueError("unsupported layer: 1 to 1024 experts, hidden and inter multiples of 32 up to 65536; got %d "
                             "experts, hidden %d, inter %d" % (experts, hidden, inter))
        block = 32 if format == "mxfp4" else 16
        self.index = w13.get_device() if w13.is_cuda else -1
        u8 = torch.uint8
        p = [_part(w13, (experts, 2 * inter, hidden // 2), u8, "w13", self.index),
             _part(w13_scales, (experts, 2 * inter, hidden // block), u8, "w13_scales", self.index),
             _part(w2, (experts, hidden, inter // 2), u8, "w2", self.index),
             _part(w2_scales, (experts, hidden, inter // block), u8, "w2_scales", self.index)]
        if format == "mxfp4":
            if w13_scale2 is not None or w2_scale2 is not None:
                raise ValueError("mxfp4 has no scale2")
            p += [None, None]
        else:
            p += [_part(w13_scale2, (experts,), torch.float32, "w13_scale2", self.index),
                  _part(w2_scale2, (experts,), torch.float32, "w2_scale2", self.index)]
        if router is not None:
            if (router.experts, router.hidden) != (experts, hidden):
                raise ValueError("the router has %d experts and hidden %d, the layer %d and %d"
                                 % (router.experts, router.hidden, experts, hidden))
            if router.index != self.index:
                raise ValueError("the router is on another device than the layer")
        self.format, self._router, self.experts, self.hidden, self.inter = format, router, experts, hidden, inter
        self._w13, self._w13_scales, self._w2, self._w2_scales = w13, w13_scales, w2, w2_scales
        self._w13_scale2, self._w2_scale2 = w13_scale2, w2_scale2
        _moe_lib()
        self._handle = bytes(_CWeights(MOE_FORMATS[format], experts, hidden, inter, *p))


def moe_nbytes(router: Optional[MoERouter], layer: Optional[MoE], tokens: int, top_k: int) -> int:
    """Bytes of workspace of moe_route (layer None), moe_experts (router None) or moe; -1 if invalid."""
    r = None if router is None else ctypes.byref(_CRouter.from_buffer_copy(router._handle))
    w = None if layer is None else ctypes.byref(_CWeights.from_buffer_copy(layer._handle))
    return int(_moe_lib().qbn_moe_workspace(r, w, tokens, top_k))


def moe_route(router: MoERouter, x: torch.Tensor, ids: Optional[torch.Tensor] = None,
              weights: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The experts of each row of x (bfloat16 [tokens][hidden]), best first, equal
    ones by their number: (ids int32 [tokens][top_k], weights float32 [tokens][top_k])."""
    got = (kv._calls or kv._call()).moe_route(router._handle, router.index, x, ids, weights, workspace)
    if got.__class__ is int:
        raise QbnError(got, "qbn_moe_route")
    return got


def moe_experts(layer: MoE, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Sum over a token's experts (ids int32 [tokens][top_k]; one that is no
    expert's number stands for none) of weight * W2 (silu(gate x) * (up x)), bfloat16
    [tokens][hidden]."""
    got = (kv._calls or kv._call()).moe_experts(layer._handle, layer.index, x, ids, weights, out, workspace)
    if got.__class__ is int:
        raise QbnError(got, "qbn_moe_experts")
    return got


def moe(layer: MoE, x: torch.Tensor, out: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
        weights: Optional[torch.Tensor] = None,
        workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The whole layer for x (bfloat16 [tokens][hidden]): moe_route and moe_experts
    in one call. (out bfloat16 [tokens][hidden], ids, weights)."""
    if layer._router is None:
        raise ValueError("the layer has no router: use moe_experts")
    got = (kv._calls or kv._call()).moe(layer._router._handle, layer._handle, layer.index, x, out, ids, weights, workspace)
    if got.__class__ is int:
        raise QbnError(got, "qbn_moe")
    return got
