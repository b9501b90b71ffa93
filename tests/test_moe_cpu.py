"""Host-side tests of the experts' layer that need no GPU: exports, struct sizes,
workspaces, refusals (no pointer below is dereferenced: every call fails its
checks or has nothing to do), and pins of the test reference."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import step_ref as S
from bit_block_quantized_nibble_amd import experts, kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, FORMAT, UNSUP, SHAPE, ALIGN, SCALE2, NANS, DTYPE, HIP, GROUP = range(11)
A, B = 0x10000, 0x9000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return experts._moe_lib()


def router(n=8, top=2, hidden=64, normalize=1, weight=A, bias=None):
    return ctypes.byref(experts._CRouter(n, top, hidden, normalize, weight, bias))


def weights(format=1, n=8, hidden=64, inter=32, w13=A, s13=A, w2=A, s2=A, f13=None, f2=None):
    return ctypes.byref(experts._CWeights(format, n, hidden, inter, w13, s13, w2, s2, f13, f2))


def test_exports_every_declared_symbol(lib):
    header = open(os.path.join(ROOT, "include", "qbn_moe.h")).read()
    declared = re.findall(r"QBN_API\s+[\w\s\*]+?\b(qbn_\w+)\s*\(", header)
    assert set(declared) == set(experts.MOE_EXPORTED) and len(declared) == len(experts.MOE_EXPORTED)
    for name in declared:
        assert hasattr(ctypes.CDLL(qbn.lib_path()), name), name
    assert [lib.qbn_moe_struct_size(i) for i in range(3)] == [32, 64, 0]


BAD_ROUTERS = [(dict(n=0), SHAPE), (dict(n=1025), SHAPE), (dict(top=0), SHAPE), (dict(top=9), SHAPE),
               (dict(n=64, top=33), SHAPE), (dict(hidden=48), SHAPE), (dict(hidden=0), SHAPE),
               (dict(hidden=(1 << 16) + 32), SHAPE), (dict(normalize=2), FORMAT)]
BAD_ROUTER_PARTS = [(dict(weight=None), NULL), (dict(weight=A + 8), ALIGN), (dict(bias=A + 2), ALIGN)]
BAD_WEIGHTS = [(dict(format=3), UNSUP), (dict(format=8), UNSUP), (dict(format=0), FORMAT), (dict(format=99), FORMAT),
               (dict(n=0), SHAPE), (dict(n=1025), SHAPE), (dict(hidden=40), SHAPE), (dict(inter=48), SHAPE),
               (dict(inter=-32), SHAPE), (dict(inter=(1 << 16) + 32), SHAPE)]
BAD_WEIGHT_PARTS = [(dict(w13=None), NULL), (dict(s13=None), NULL), (dict(w2=None), NULL), (dict(s2=None), NULL),
                    (dict(w13=A + 4), ALIGN), (dict(s13=A + 1), ALIGN), (dict(w2=A + 8), ALIGN), (dict(s2=A + 2), ALIGN),
                    (dict(f13=A), SCALE2), (dict(f2=A), SCALE2), (dict(format=2), NULL), (dict(format=2, f13=A), NULL),
                    (dict(format=2, f13=A + 2, f2=A), ALIGN)]


def test_refusals_of_layers(lib):
    def route(r):
        return lib.qbn_moe_route(r, 3, A, 64, A, A, A, BIG, None)

    def apply(w):
        return lib.qbn_moe_experts(w, 3, 2, A, 64, A, A, B, 64, A, BIG, None)

    def both(r, w):
        return lib.qbn_moe(r, w, 3, A, 64, A, A, B, 64, A, BIG, None)

    assert route(None) == apply(None) == both(None, weights()) == both(router(), None) == NULL
    for kw, want in BAD_ROUTERS + BAD_ROUTER_PARTS:
        assert route(router(**kw)) == both(router(**kw), weights()) == want, kw
    for kw, want in BAD_WEIGHTS + BAD_WEIGHT_PARTS:
        assert apply(weights(**kw)) == both(router(), weights(**kw)) == want, kw
    for kw in (dict(n=7), dict(hidden=32)):
        assert both(router(**kw), weights()) == SHAPE, kw


def test_refusals_of_arguments(lib):
    def call(which, tokens=3, top=2, x=A, xs=64, ids=A, w=A, out=B, os=64, ws=A, wsb=BIG):
        if which == "route":
            return lib.qbn_moe_route(router(), tokens, x, xs, ids, w, ws, wsb, None)
        if which == "experts":
            return lib.qbn_moe_experts(weights(), tokens, top, x, xs, ids, w, out, os, ws, wsb, None)
        return lib.qbn_moe(router(), weights(), tokens, x, xs, ids, w, out, os, ws, wsb, None)

    for which in ("route", "experts", "both"):
        for kw, want in [(dict(tokens=-1), SHAPE), (dict(tokens=(1 << 24) + 1), SHAPE), (dict(x=None), NULL),
                         (dict(x=A + 8), ALIGN), (dict(xs=56), SHAPE), (dict(xs=-64), SHAPE), (dict(xs=68), ALIGN),
                         (dict(xs=1 << 31), SHAPE), (dict(ids=None), NULL), (dict(ids=A + 1), ALIGN), (dict(w=None), NULL),
                         (dict(w=A + 2), ALIGN), (dict(ws=None), NULL), (dict(ws=A + 8), ALIGN), (dict(wsb=7), SHAPE)]:
            assert call(which, **kw) == want, (which, kw)
        assert call(which, tokens=0, x=None, ids=None, w=None, out=None, ws=None, wsb=0) == OK
        if which != "route":
            for kw, want in [(dict(out=None), NULL), (dict(out=B + 2), ALIGN), (dict(os=63), SHAPE), (dict(os=68), ALIGN),
                             (dict(out=A), UNSUP), (dict(out=A + 16), UNSUP), (dict(out=A + 2 * 3 * 64 - 16), UNSUP)]:
                assert call(which, **kw) == want, (which, kw)
    for top in (0, -1, 33):
        assert call("experts", top=top) == SHAPE


def test_workspaces(lib):
    f = lib.qbn_moe_workspace
    assert f(None, None, 1, 1) == -1 and f(router(n=0), None, 1, 1) == -1 and f(None, weights(format=4), 1, 1) == -1
    assert f(router(), None, -1, 1) == -1 and f(router(), None, 1, 0) == -1 and f(router(), None, 1, 33) == -1
    assert f(router(), weights(), (1 << 24) + 1, 2) == -1 and f(router(), None, 0, 2) == 0 and f(None, weights(), 0, 2) == 0
    for t in (1, 5, 32, 33, 100, 256, 1000, 5000):
        a, b = f(router(), None, t, 2), f(None, weights(), t, 2)
        assert a >= 8 * 8 * min(t, 4096) and b >= 2 * min(t, 256) * 4 * 32 and f(router(), weights(), t, 2) == a + b
        assert a % 16 == 0 and b % 16 == 0
    # a portion of tokens at a time: it stops growing
    assert f(None, weights(), 256, 2) == f(None, weights(), 1 << 24, 2)


def test_handles_refuse_host_tensors_and_other_sizes():
    bf, u8 = torch.bfloat16, torch.uint8
    with pytest.raises(ValueError, match="device"):
        qbn.MoERouter(torch.zeros(4, 64, dtype=bf), 2)
    with pytest.raises(TypeError, match="dtype"):
        qbn.MoERouter(torch.zeros(4, 64), 2)
    for shape, top in (((4, 64), 5), ((4, 64), 0), ((4, 40), 2), ((1025, 32), 2), ((64, 64), 33)):
        with pytest.raises(ValueError, match="unsupported router"):
            qbn.MoERouter(torch.zeros(shape, dtype=bf), top)
    with pytest.raises(ValueError):
        qbn.MoERouter(torch.zeros(4, dtype=bf), 1)
    z = lambda *s: torch.zeros(s, dtype=u8)  # noqa: E731
    with pytest.raises(ValueError, match="format"):
        qbn.MoE("q4_0", None, z(2, 64, 32), z(2, 64, 2), z(2, 64, 16), z(2, 64, 1))
    with pytest.raises(ValueError, match="device"):
        qbn.MoE("mxfp4", None, z(2, 64, 32), z(2, 64, 2), z(2, 64, 16), z(2, 64, 1))
    with pytest.raises(ValueError, match="unsupported layer"):
        qbn.MoE("mxfp4", None, z(2, 48, 32), z(2, 48, 2), z(2, 64, 12), z(2, 64, 1))
    with pytest.raises(ValueError, match="w13 must be"):
        qbn.MoE("mxfp4", None, z(2, 64, 16), z(2, 64, 2), z(2, 64, 16), z(2, 64, 1))


def test_call_module_checks():
    call = kv._call()
    r, w = bytes(experts._CRouter(8, 2, 64, 1, A, None)), bytes(experts._CWeights(1, 8, 64, 32, A, A, A, A, None, None))
    x, ids, ww = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    for a, error, words in [
            ((r, 0, x, None, None, None), ValueError, "x is on cpu, the layer on another device"),
            ((r, -1, x.float(), None, None, None), TypeError, "x dtype"),
            ((r, -1, x[0], None, None, None), ValueError, r"x must be \[tokens\]\[64\]"),
            ((r, -1, x[:, :32], None, None, None), ValueError, "x must be"),
            ((r, -1, x, ids.long(), None, None), TypeError, "ids dtype"),
            ((r, -1, x, ids[:2], None, None), ValueError, "ids must be"),
            ((r, -1, x, ids, ww[:, :1], None), ValueError, "weights must be"),
            ((r, -1, x, ids, ww.double(), None), TypeError, "weights dtype"),
            ((r, -1, x, ids, ww, torch.zeros(1)), ValueError, "workspace holds 4 bytes"),
            ((w, -1, x, None, None, None), TypeError, "not a handle"),
            ((r, -1, x), TypeError, "wanted")]:
        with pytest.raises(error, match=words):
            call.moe_route(*a)
    for a, error, words in [
            ((w, -1, x, None, ww, None, None), TypeError, "ids and weights"),
            ((w, -1, x, ids, ww[:2], None, None), ValueError, "weights must be"),
            ((w, -1, x, ids[0], ww, None, None), ValueError, "ids must be"),
            ((w, -1, x, ids, ww, x[:2], None), ValueError, "out must be"),
            ((w, -1, x, ids, ww, x.float(), None), TypeError, "out dtype"),
            ((w, 0, x, ids, ww, None, None), ValueError, "another device")]:
        with pytest.raises(error, match=words):
            call.moe_experts(*a)
    with pytest.raises(TypeError, match="wanted"):
        call.moe(r, w)
    with pytest.raises(ValueError, match="out must be"):
        call.moe(r, w, -1, x, x[:1], None, None, None)


def test_reference_layer_one_number_at_a_time():
    """The reference of the GPU tests against loops over single numbers."""
    rng = np.random.default_rng(0)
    c13, s13, _, c2, s2, _ = S.layer(rng, "mxfp4", 2, 32, 32)
    w13, w2 = S.decode("mxfp4", c13, s13), S.decode("mxfp4", c2, s2)
    grid = [0, .5, 1, 1.5, 2, 3, 4, 6]
    for e, r, k in ((0, 0, 0), (1, 63, 31), (0, 17, 12)):
        code = int(c13[e, r, k // 2]) >> (4 * (k % 2)) & 15
        assert w13[e, r, k] == (-1) ** (code >> 3) * grid[code & 7] * 2.0 ** (int(s13[e, r, k // 32]) - 127)
    x, ids, ww = rng.standard_normal((1, 32)), np.array([[1, -1]]), np.array([[0.25, 9.0]])
    out, tol = S.experts(x, ids, ww, w13, w2)
    h = []
    for i in range(32):
        g, u = sum(w13[1, i] * x[0]), sum(w13[1, 32 + i] * x[0])
        h.append(g / (1 + np.exp(-g)) * u)
    assert np.allclose(out[0], [0.25 * sum(w2[1, n] * np.array(h)) for n in range(32)], rtol=1e-12)
    assert (tol > 0).all()


def test_reference_choice():
    x, w = np.eye(4)[:2], np.array([[1, 5, 0, 0], [2, 5, 0, 0], [1, 7, 0, 0.]])
    ids, share, gap = S.route(x, w, None, 2, True)
    assert ids.tolist() == [[1, 0], [2, 0]] and np.allclose(share.sum(1), 1) and gap == 0.0
    assert np.allclose(share[0], np.exp([2, 1]) / np.exp([2, 1]).sum())
    _, share, _ = S.route(x, w, np.zeros(3), 2, False)
    assert np.allclose(share[0], np.exp([2, 1]) / np.exp([1, 2, 1]).sum())
