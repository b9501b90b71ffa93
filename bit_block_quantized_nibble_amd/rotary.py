"""Rotary positions: binding of include/qbn_rope.h.

`Rope` holds a model's rotation (frequencies as fractions of a turn, in device
memory), `rope` turns vectors by their positions, and `kv_append_rope` does
it on the way into a paged cache. As in the rest of the package nothing is
computed here but the frequencies, once: what the C ABI cannot see (devices,
dtypes, sizes) is checked, and pointers are passed.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Union

import torch

from . import QbnError, _load, kv
from .kv import KVCache, _fixed

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_EXPORTED = ("qbn_rotation_struct_size", "qbn_rope", "qbn_kv_append_rope")
_TWO_PI = 628318530717958647692528676655900576839433879875021164194988918  # 10^62 of it
_ONE = 10 ** 62 << 64


class _CRotation(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rot", ctypes.c_int32), ("factor", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_void_p)]


_bound = None


def _rope_lib():
    """libqbn with the argument types of the rotation's entry points."""
    global _bound
    if _bound is not None:
        return _bound
    lib = _load()
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    R, C, B = ctypes.POINTER(_CRotation), ctypes.POINTER(kv._CCache), ctypes.POINTER(kv._CBatch)
    lib.qbn_rotation_struct_size.argtypes, lib.qbn_rotation_struct_size.restype = [], ctypes.c_size_t
    for name, args in (
            ("qbn_rope", [R, I64, I32, I32, P, P, I64, I64, P, I64, I64, I32, P]),
            ("qbn_kv_append_rope", [C, I64, B, R, I32, P, I64, I64, P, I64, I64, P, I64, I64, P, I64, I64, I32, P])):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, I32
    if lib.qbn_rotation_struct_size() != ctypes.sizeof(_CRotation):
        raise RuntimeError("libqbn ABI mismatch: rebuild the library")
    _bound = lib
    return lib


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", scale: float = 1.0,
                     original: float = 0.0, low: float = 1.0, high: float = 4.0, fast: float = 32.0,
                     slow: float = 1.0):
    """(frequencies in radians per position, rot / 2 of them; factor on cosine and
    sine). f_i = base^(-2 i / rot), for contexts `scale` times as long as the
    `original` (trained) one changed by `scaling`:

    none    f_i.
    linear  f_i / scale.
    ntk     base * scale^(rot / (rot - 2)) in base's place.
    bands   by the turns n = original * f_i / 2 pi in the trained length: f_i from
            `high` turns on, f_i / scale up to `low`, and between them
            p f_i + (1 - p) f_i / scale with p = (n - low) / (high - low).
    yarn    the same with p = 1 - clamp((i - a) / (b - a)), where a and b are the
            pairs (rounded outwards, in 0 .. rot - 1) that make `fast` and `slow`
            turns; the factor is 0.1 ln scale + 1, and 1 where scale is no more than 1.
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be a positive even number")
    if scaling not in ("none", "linear", "ntk", "bands", "yarn"):
        raise ValueError("unknown scaling %r" % (scaling,))
    if not (base > 0 and math.isfinite(base) and scale > 0 and math.isfinite(scale)):
        raise ValueError("base and scale must be positive")
    if scaling in ("bands", "yarn") and not (original > 0 and math.isfinite(original)):
        raise ValueError("%s needs the original context length" % scaling)
    factor = 1.0
    if scaling == "ntk":
        if rot <= 2:
            raise ValueError("ntk needs rot > 2")
        base = base * scale ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / scale for x in f]
    elif scaling == "bands":
        if not high > low:
            raise ValueError("high must be above low")
        part = [min(1.0, max(0.0, (original * x / (2 * math.pi) - low) / (high - low))) for x in f]
        f = [x * p + x / scale * (1 - p) for x, p in zip(f, part)]
    elif scaling == "yarn":
        if base == 1.0 or not (fast > 0 and slow > 0):
            raise ValueError("yarn needs a base other than 1 and positive numbers of turns")
        a, b = (rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow))
        a, b = max(0, math.floor(a)), min(rot - 1, math.ceil(b))
        part = [min(1.0, max(0.0, (i - a) / max(b - a, 0.001))) for i in range(rot // 2)]
        f = [x * (1 - p) + x / scale * p for x, p in zip(f, part)]
        factor = 0.1 * math.log(scale) + 1.0 if scale > 1 else 1.0
    return f, factor


def _turns(frequency: float) -> int:
    """The frequency in whole turns of 2^64 parts, to the nearest part (ties, which an
    irrational number's multiples do not have, aside), as the int64 of the same bits."""
    n, d = frequency.as_integer_ratio()
    d *= _TWO_PI
    return ((2 * n * _ONE + d) // (2 * d) + (1 << 63) & (1 << 64) - 1) - (1 << 63)


class Rope:
    """A rotation by positions: `frequencies` (radians per position, one for each
    of the rot / 2 pairs, any sequence of numbers; taken in binary64), the layout
    of the pairs ("half": element i with i + rot / 2, "interleaved": 2 i with
    2 i + 1) and the factor on cosine and sine. One made on the host (device "cpu")
    holds its turns there and turns nothing: rope and kv_append_rope refuse it."""

    turns = _fixed("turns", "Turns per position of each pair, in units of 2^-64 (int64 of the same bits).")

    def __init__(self, frequencies: Union[Sequence[float], torch.Tensor], layout: str = "half", factor: float = 1.0,
                 device="cuda"):
        if layout not in ROPE_LAYOUTS:
            raise ValueError("unknown layout %r" % (layout,))
        if isinstance(frequencies, torch.Tensor):
            frequencies = frequencies.double().reshape(-1).tolist()
        f = [float(x) for x in frequencies]
        if not f or len(f) % 8:
            raise ValueError("%d frequencies: a positive multiple of 8 is wanted (rot a multiple of 16)" % len(f))
        if not all(math.isfinite(x) for x in f) or not math.isfinite(factor):
            raise ValueError("frequencies and factor must be finite")
        self._turns = torch.tensor([_turns(x) for x in f], dtype=torch.int64, device=device)
        self.layout, self.rot, self.factor, self.frequencies = layout, 2 * len(f), float(factor), f
        self.index = self._turns.get_device() if self._turns.is_cuda else -1
        _rope_lib()
        self._handle = bytes(_CRotation(ROPE_LAYOUTS[layout], self.rot, self.factor, 0, self._turns.data_ptr()))

    @classmethod
    def make(cls, rot: int, base: float = 10000.0, scaling: str = "none", layout: str = "half", device="cuda",
             **more) -> "Rope":
        """The rotation with rope_frequencies(rot, base, scaling, **more) and its factor."""
        f, factor = rope_frequencies(rot, base, scaling, **more)
        return cls(f, layout, factor, device)


def rope(x: torch.Tensor, positions: torch.Tensor, rotation: Rope, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [tokens][heads][dim] (float32 or bfloat16, the last axis contiguous) with
    the first rotation.rot elements of every head turned by the token's position
    (int32 [tokens]). out: another tensor of the same sizes and dtype, or x itself
    to turn it in its place."""
    got = (kv._calls or kv._call()).rope(rotation._handle, rotation.index, x, positions, out)
    if got.__class__ is int:
        raise QbnError(got, "qbn_rope")
    return got


def kv_append_rope(cache: KVCache, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, table: torch.Tensor,
                   lens: torch.Tensor, rotation: Rope, cu: Optional[torch.Tensor] = None, layer: int = 0,
                   out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """kv_append with the keys turned by their positions in their sequences (the
    last new token's is lens - 1) before they are stored. q [tokens][q_heads]
    [head_dim], of k's dtype, is turned alike and returned as bfloat16 (`out`, or q
    itself to turn it in its place, or a new tensor); None without q. Rows of no
    sequence are not stored, and their q is copied as it is."""
    got = (kv._calls or kv._call()).append_rope(cache._handle, cache.index, q, k, v, table, lens, cu, layer,
                                                rotation._handle, rotation.index, out)
    if got.__class__ is int:
        raise QbnError(got, "qbn_kv_append_rope")
    return got
