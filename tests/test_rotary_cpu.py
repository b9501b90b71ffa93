"""Host-side tests of the rotation by positions that need no GPU: exports, struct
size, refusals (no pointer below is dereferenced: every call fails its checks or
has nothing to do), the frequencies and their fractions of a turn."""
import ctypes
import math
import os
import re
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import step_ref as S
from bit_block_quantized_nibble_amd import kv, rotary

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, FORMAT, UNSUP, SHAPE, ALIGN, SCALE2, NANS, DTYPE, HIP, GROUP = range(11)
A, B = 0x10000, 0x9000000
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    return rotary._rope_lib()


def rotation(layout=0, rot=64, factor=1.0, reserved=0, turns=A):
    return ctypes.byref(rotary._CRotation(layout, rot, factor, reserved, turns))


def cache(format=16, heads=2, dim=64, page=16, layers=1, pages=8):
    return ctypes.byref(kv._CCache(format, heads, dim, page, layers, pages, A, A, A, A))


def batch(seqs=4, tokens=4, row=8, table=A, lens=A, cu=None):
    return ctypes.byref(kv._CBatch(seqs, tokens, row, row, table, lens, cu))


def test_exports_every_declared_symbol(lib):
    header = open(os.path.join(ROOT, "include", "qbn_rope.h")).read()
    declared = re.findall(r"QBN_API\s+[\w\s\*]+?\b(qbn_\w+)\s*\(", header)
    assert set(declared) == set(rotary.ROPE_EXPORTED) and len(declared) == len(rotary.ROPE_EXPORTED)
    for name in declared:
        assert hasattr(ctypes.CDLL(qbn.lib_path()), name), name
    assert lib.qbn_rotation_struct_size() == ctypes.sizeof(rotary._CRotation) == 24


def call_rope(lib, r=None, tokens=4, heads=2, dim=64, pos=A, x=A, xt=128, xh=64, out=B, ot=128, oh=64, dtype=BF16):
    return lib.qbn_rope(rotation() if r is None else r, tokens, heads, dim, pos, x, xt, xh, out, ot, oh, dtype, None)


BAD_ROTATIONS = [(dict(layout=2), FORMAT), (dict(layout=-1), FORMAT), (dict(reserved=1), FORMAT), (dict(rot=0), SHAPE),
                 (dict(rot=24), SHAPE), (dict(rot=-16), SHAPE), (dict(rot=80), SHAPE), (dict(factor=math.inf), SHAPE),
                 (dict(factor=math.nan), SHAPE), (dict(turns=None), NULL), (dict(turns=A + 8), ALIGN)]


def test_rope_refusals(lib):
    assert lib.qbn_rope(None, 4, 2, 64, A, A, 128, 64, B, 128, 64, BF16, None) == NULL
    for kw, want in BAD_ROTATIONS:
        assert call_rope(lib, rotation(**kw)) == want, kw
    for kw, want in [(dict(dim=72), SHAPE), (dict(dim=0), SHAPE), (dict(dim=1040), SHAPE), (dict(tokens=-1), SHAPE),
                     (dict(heads=-1), SHAPE), (dict(heads=(1 << 16) + 1), SHAPE), (dict(tokens=(1 << 30) + 1), SHAPE),
                     (dict(dtype=3), FORMAT), (dict(dtype=2), DTYPE), (dict(pos=None), NULL), (dict(pos=A + 2), ALIGN),
                     (dict(x=None), NULL), (dict(x=A + 8), ALIGN), (dict(xt=-128), SHAPE), (dict(xt=1 << 60), SHAPE),
                     (dict(xh=4), ALIGN), (dict(out=None), NULL), (dict(out=B + 2), ALIGN), (dict(ot=132), ALIGN),
                     (dict(ot=0), SHAPE), (dict(ot=64), SHAPE), (dict(oh=0), SHAPE), (dict(oh=56), SHAPE),
                     (dict(out=A + 16), UNSUP), (dict(out=A, ot=256), UNSUP), (dict(out=A + 2 * 3 * 128), UNSUP)]:
        assert call_rope(lib, **kw) == want, kw
    # nothing to do
    assert call_rope(lib, tokens=0, pos=None, x=None, out=None) == OK
    assert call_rope(lib, heads=0, pos=None, x=None, out=None) == OK


def call_append(lib, c=None, b=None, r=None, layer=0, qh=4, q=A, qo=B, ot=256, oh=64, k=A, v=A, dtype=BF16, qs=(256, 64)):
    return lib.qbn_kv_append_rope(cache() if c is None else c, layer, batch() if b is None else b,
                                  rotation() if r is None else r, qh, q, *qs, qo, ot, oh, k, 128, 64, v, 128, 64, dtype, None)


def test_append_refusals(lib):
    assert lib.qbn_kv_append_rope(None, 0, batch(), rotation(), 0, None, 0, 0, None, 0, 0, A, 128, 64, A, 128, 64, 1, None) == NULL
    for kw, want in BAD_ROTATIONS:
        assert call_append(lib, r=rotation(**kw)) == want, kw
    for kw, want in [(dict(c=cache(format=2)), FORMAT), (dict(c=cache(dim=80)), UNSUP), (dict(b=batch(tokens=3)), SHAPE),
                     (dict(b=batch(lens=None)), NULL), (dict(b=batch(table=None)), NULL), (dict(layer=1), SHAPE),
                     (dict(dtype=2), DTYPE), (dict(dtype=5), FORMAT), (dict(qh=-1), SHAPE), (dict(qh=(1 << 16) + 1), SHAPE),
                     (dict(q=None), NULL), (dict(qo=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
                     (dict(k=A + 4), ALIGN), (dict(v=A + 2), ALIGN), (dict(q=A + 8), ALIGN), (dict(qo=B + 8), ALIGN),
                     (dict(ot=0), SHAPE), (dict(oh=32), SHAPE), (dict(qo=A + 64), UNSUP),
                     (dict(qo=A, ot=512), UNSUP),                     # q's place, other strides
                     (dict(q=B, qo=A), UNSUP),                        # over k
                     (dict(q=A, qo=A, dtype=F32), UNSUP)]:            # other element sizes
        assert call_append(lib, **kw) == want, kw
    empty = batch(seqs=0, tokens=0)
    assert call_append(lib, b=empty, q=None, qo=None, k=None, v=None) == OK


def test_call_module_checks():
    call = kv._call()
    r = bytes(rotary._CRotation(0, 64, 1.0, 0, A))
    c = bytes(kv._CCache(16, 2, 64, 16, 1, 8, A, A, A, A))
    x, pos = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32)
    t, cu = torch.zeros(4, 8, dtype=torch.int32), None
    for a, error, words in [
            ((r, 0, x, pos, None), ValueError, "x is on cpu, the rotation on another device"),
            ((r, -1, x[0], pos, None), ValueError, r"x must be \[tokens\]\[heads\]\[dim\]"),
            ((r, -1, x.half(), pos, None), TypeError, "x dtype"),
            ((r, -1, x, pos.long(), None), TypeError, "positions dtype"),
            ((r, -1, x, pos[:3], None), ValueError, "positions has 3 entries"),
            ((r, -1, x, None, None), TypeError, "positions must be a tensor"),
            ((r, -1, x, pos, x[:3]), ValueError, "out must be"),
            ((r, -1, x, pos, x.bfloat16()), TypeError, "out dtype"),
            ((r, -1, x.transpose(1, 2), pos, None), ValueError, "last axis of x"),
            ((r, -1, x, pos, torch.zeros(4, 64, 2).transpose(1, 2)), ValueError, "last axis of out"),
            ((b"no", -1, x, pos, None), TypeError, "not a handle"),
            ((r, -1, x, pos), TypeError, "wanted")]:
        with pytest.raises(error, match=words):
            call.rope(*a)
    ok = dict(c=c, dev=-1, q=x, k=x, v=x, table=t, lens=pos, cu=cu, layer=0, r=r, rdev=-1, out=None)
    for kw, error, words in [
            (dict(dev=0, rdev=0), ValueError, "another device"), (dict(rdev=0), ValueError, "another device"),
            (dict(k=x[:, :1]), ValueError, "k must be"), (dict(v=x[:3]), ValueError, "alike"),
            (dict(q=x[:3]), ValueError, "q and k must be alike"), (dict(q=x.bfloat16()), ValueError, "q and k must be alike"),
            (dict(q=None, out=x), ValueError, "None"), (dict(out=x), TypeError, "out dtype"),
            (dict(k=x.double(), v=x.double()), TypeError, "k dtype"), (dict(lens=pos[:3]), ValueError, "lens has 3"),
            (dict(table=t.long()), TypeError, "table dtype"), (dict(r=b"no"), TypeError, "not a handle")]:
        a = dict(ok)
        a.update(kw)
        with pytest.raises(error, match=words):
            call.append_rope(*a.values())


def test_rope_object_checks():
    for bad in ([], [1.0] * 7, [1.0] * 12):
        with pytest.raises(ValueError, match="frequencies"):
            qbn.Rope(bad, device="cpu")
    with pytest.raises(ValueError, match="finite"):
        qbn.Rope([math.nan] * 8, device="cpu")
    with pytest.raises(ValueError, match="finite"):
        qbn.Rope([1.0] * 8, factor=math.inf, device="cpu")
    with pytest.raises(ValueError, match="layout"):
        qbn.Rope([1.0] * 8, layout="neither", device="cpu")
    r = qbn.Rope(torch.ones(8), device="cpu")
    with pytest.raises(AttributeError, match="fixed"):
        r.turns = torch.zeros(8, dtype=torch.int64)
    assert r.rot == 16 and r.frequencies == [1.0] * 8


def test_fractions_of_a_turn():
    """round(f / 2 pi * 2^64) mod 2^64, against a decimal computation."""
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    f = [1.0, 0.1, 1e-5, 6.283185307179586, 100.0, -0.25, 0.0, 10000.0 ** (-62 / 64)]
    got = [int(t) % (1 << 64) for t in qbn.Rope(f, device="cpu").turns.tolist()]
    want = [int((Decimal(x) / (2 * pi) * (1 << 64)).to_integral_value()) % (1 << 64) for x in f]
    assert got == want


def test_frequencies():
    plain, one = qbn.rope_frequencies(64, 10000.0)
    assert one == 1.0 and np.allclose(plain, 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    f, one = qbn.rope_frequencies(64, 10000.0, "linear", scale=4.0)
    assert one == 1.0 and np.allclose(f, np.array(plain) / 4, rtol=1e-15)
    # ntk: the lowest frequency is stretched by the scale, the highest not at all
    f, _ = qbn.rope_frequencies(64, 10000.0, "ntk", scale=4.0)
    assert f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 4, rel_tol=1e-12)
    f, _ = qbn.rope_frequencies(64, 10000.0, "bands", scale=8.0, original=8192, low=1.0, high=4.0)
    for a, b in zip(f, plain):
        turns = 8192 * b / (2 * math.pi)
        assert (a == b) if turns >= 4 else math.isclose(a, b / 8, rel_tol=1e-14) if turns <= 1 else b / 8 < a < b
    f, factor = qbn.rope_frequencies(64, 10000.0, "yarn", scale=16.0, original=4096)
    assert math.isclose(factor, 0.1 * math.log(16) + 1)
    assert f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 16, rel_tol=1e-12)
    assert all(b / 16 * (1 - 1e-12) <= a <= b for a, b in zip(f, plain)) and all(a > b for a, b in zip(f, f[1:]))
    for kw in (dict(scaling="other"), dict(scale=0.0), dict(base=-1.0), dict(scaling="bands"), dict(scaling="yarn"),
               dict(scaling="bands", original=8.0, low=2.0, high=2.0), dict(base=math.inf)):
        with pytest.raises(ValueError):
            qbn.rope_frequencies(64, **kw)
    with pytest.raises(ValueError):
        qbn.rope_frequencies(7)


def test_reference_turns_by_complex_numbers():
    """The reference of the GPU tests against products of complex numbers."""
    rng = np.random.default_rng(0)
    x, pos, f = rng.standard_normal((3, 2, 40)), np.array([0, 7, 12345]), 10000.0 ** (-np.arange(16) / 16)
    for layout in ("half", "interleaved"):
        y, tol = S.turn(x, pos, f, layout, 1.5)
        z = x[..., :16] + 1j * x[..., 16:32] if layout == "half" else x[..., 0:32:2] + 1j * x[..., 1:32:2]
        z = z * 1.5 * np.exp(1j * np.outer(pos, f))[:, None]
        got = y[..., :16] + 1j * y[..., 16:32] if layout == "half" else y[..., 0:32:2] + 1j * y[..., 1:32:2]
        assert np.abs(got - z).max() < 1e-10 and np.array_equal(y[..., 32:], x[..., 32:]) and tol.max() < 1e-4
