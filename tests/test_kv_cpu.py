"""Host-side tests of the paged key-value cache that need no GPU: exports,
struct sizes, refusals of the C ABI (no pointer below is dereferenced: every
call fails its checks or has nothing to do), the binding's own checks, and
pins of the test reference."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
from bit_block_quantized_nibble_amd import kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, FORMAT, UNSUP, SHAPE, ALIGN, SCALE2, NANS, DTYPE, HIP, GROUP = range(11)
A, B = 0x10000, 0x9000000


@pytest.fixture(scope="module")
def lib():
    return kv._kv()


def cache(format=16, heads=2, dim=64, page=16, layers=1, pages=8, k=A, v=A, ks=A, vs=A):
    return ctypes.byref(kv._CCache(format, heads, dim, page, layers, pages, k, v, ks, vs))


def batch(seqs=4, tokens=4, row=8, stride=None, table=A, lens=A, cu=None):
    return ctypes.byref(kv._CBatch(seqs, tokens, row, row if stride is None else stride, table, lens, cu))


def pool(seqs=4, row=8, pages=8, page=16, reserved=0, table=A, lens=A + 0x1000, refs=A + 0x2000):
    return ctypes.byref(kv._CPool(seqs, row, pages, page, reserved, table, lens, refs))


def test_exports_every_declared_symbol(lib):
    header = open(os.path.join(ROOT, "include", "qbn_kv.h")).read()
    declared = re.findall(r"QBN_API\s+[\w\s\*]+?\b(qbn_\w+)\s*\(", header)
    assert set(declared) == set(kv.KV_EXPORTED) and len(declared) == len(kv.KV_EXPORTED)
    for name in declared:
        assert hasattr(ctypes.CDLL(qbn.lib_path()), name), name
    assert [lib.qbn_kv_struct_size(i) for i in range(4)] == [64, 56, 56, 0]


def test_bytes(lib):
    assert qbn.kv_nbytes("bf16", 2, 10, 8, 64, 128) == 2 * 10 * 8 * 64 * 128 * 2
    assert qbn.kv_nbytes("bf16", 2, 10, 8, 64, 128, 1) == 0
    assert qbn.kv_nbytes("mxfp4", 1, 10, 8, 64, 128) + qbn.kv_nbytes("mxfp4", 1, 10, 8, 64, 128, 1) == 10 * 8 * 64 * 68
    assert qbn.kv_nbytes("mxfp8", 1, 1, 1, 16, 96) == 16 * 96 and qbn.kv_nbytes("mxfp8", 1, 1, 1, 16, 96, 1) == 48
    for bad in ((1, 10, 8, 24, 128), (1, 10, 8, 64, 80), (0, 10, 8, 64, 128), (1, 0, 8, 64, 128), (1, 10, 0, 64, 128),
                (1, 1 << 31, 8, 64, 128), (1 << 20, 1 << 30, 8, 64, 128)):
        assert qbn.kv_nbytes("bf16", *bad) == -1, bad
    assert lib.qbn_kv_bytes(2, 1, 1, 1, 16, 64, 0) == -1 and lib.qbn_kv_bytes(16, 1, 1, 1, 16, 64, 2) == -1


BAD_CACHES = [(dict(format=2), FORMAT), (dict(page=24), SHAPE), (dict(page=8), SHAPE), (dict(page=512), SHAPE),
              (dict(dim=80), UNSUP), (dict(heads=0), SHAPE), (dict(pages=0), SHAPE), (dict(layers=0), SHAPE),
              (dict(k=None), NULL), (dict(v=A + 8), ALIGN), (dict(format=7, ks=None), NULL),
              (dict(format=1, vs=A + 4), ALIGN), (dict(pages=1 << 40), SHAPE)]
BAD_BATCHES = [(dict(seqs=-1), SHAPE), (dict(tokens=3), SHAPE), (dict(stride=7), SHAPE), (dict(row=-1), SHAPE),
               (dict(lens=None), NULL), (dict(table=None), NULL), (dict(table=A + 2), ALIGN),
               (dict(row=1 << 27), SHAPE), (dict(seqs=0, tokens=4, cu=A), SHAPE), (dict(cu=A + 1), ALIGN)]


@pytest.mark.parametrize("which", ["append", "decode", "prefill"])
def test_refusals_of_cache_and_batch(lib, which):
    def call(c, b, layer=0):
        if which == "append":
            return lib.qbn_kv_append(c, layer, b, A, 128, 64, A, 128, 64, 1, None)
        f = lib.qbn_kv_attention_decode if which == "decode" else lib.qbn_kv_attention_prefill
        return f(c, layer, b, 4, A, 256, 64, 0.1, 0, 0, A, A, A, 1 << 40, None)

    assert call(None, batch()) == NULL and call(cache(), None) == NULL
    for kw, want in BAD_CACHES:
        assert call(cache(**kw), batch()) == want, kw
    for kw, want in BAD_BATCHES:
        assert call(cache(), batch(**kw)) == want, kw
    assert call(cache(), batch(), layer=1) == SHAPE and call(cache(), batch(), layer=-1) == SHAPE
    assert call(cache(), batch(seqs=0, tokens=0, table=None, lens=None)) == OK


def test_append_refusals(lib):
    def call(k=A, kt=128, kh=64, v=A, vt=128, vh=64, dtype=1):
        return lib.qbn_kv_append(cache(), 0, batch(), k, kt, kh, v, vt, vh, dtype, None)

    assert call(dtype=3) == FORMAT and call(dtype=2) == DTYPE
    assert call(k=None) == NULL and call(v=None) == NULL
    assert call(k=A + 8) == ALIGN and call(kt=132) == ALIGN and call(vh=68) == ALIGN
    assert call(dtype=0, kt=130) == ALIGN and call(kt=-128) == SHAPE and call(vt=1 << 60) == SHAPE


@pytest.mark.parametrize("decode", [True, False])
def test_attention_refusals(lib, decode):
    f = lib.qbn_kv_attention_decode if decode else lib.qbn_kv_attention_prefill

    def call(b=None, heads=4, q=A, qt=256, qh=64, scale=0.1, window=0, sinks=0, out=A, lse=A, ws=A, n=1 << 40):
        return f(cache(), 0, b or batch(), heads, q, qt, qh, scale, window, sinks, out, lse, ws, n, None)

    assert call(heads=3) == SHAPE and call(heads=0) == SHAPE and call(heads=1 << 17) == SHAPE
    assert call(window=-1) == SHAPE and call(sinks=-1) == SHAPE
    assert call(scale=float("nan")) == SHAPE and call(scale=float("inf")) == SHAPE
    assert call(q=None) == NULL and call(out=None) == NULL
    assert call(q=A + 8) == ALIGN and call(qt=260) == ALIGN and call(out=A + 8) == ALIGN and call(lse=A + 2) == ALIGN
    b = batch(seqs=1, tokens=1, row=4096)
    need = lib.qbn_kv_attention_workspace(cache(), b, 4, 0, 0, int(decode))
    assert need > 0
    assert call(b, ws=None) == NULL and call(b, ws=A + 8) == ALIGN and call(b, n=need - 1) == SHAPE
    assert lib.qbn_kv_attention_workspace(cache(), b, 3, 0, 0, 1) == -1
    # a short row, or a short window, needs none
    assert lib.qbn_kv_attention_workspace(cache(), batch(row=2), 4, 0, 0, int(decode)) == 0
    if decode:
        assert call(batch(cu=A)) == UNSUP


def test_pool_refusals(lib):
    def calls(a, b, n=2, rows=A, word=A, ws=A, size=1 << 40, c=None):
        c = c or cache()
        yield lib.qbn_kv_reserve(a, b, n, rows, rows, word, ws, size, None)
        yield lib.qbn_kv_fork(c, a, b, n, rows, rows, word, ws, size, None)
        yield lib.qbn_kv_free(a, b, n, rows, 0, 0, None)
        yield lib.qbn_kv_compact(c, a, b, word, ws, size, None)

    p = pool()
    for kw, want in [(dict(seqs=-1), SHAPE), (dict(row=-1), SHAPE), (dict(pages=-1), SHAPE), (dict(page=17), SHAPE),
                     (dict(reserved=1), FORMAT), (dict(pages=(1 << 20) + 1), SHAPE), (dict(table=None), NULL),
                     (dict(lens=None), NULL), (dict(refs=None), NULL), (dict(refs=A + 2), ALIGN)]:
        assert all(st == want for st in calls(pool(**kw), p)), kw
    assert all(st == NULL for st in calls(None, p)) and all(st == NULL for st in calls(p, None))
    assert all(st == SHAPE for st in calls(p, pool(row=7))) and all(st == SHAPE for st in calls(p, pool(page=32)))
    # partly shared or overlapping tables
    assert all(st == UNSUP for st in calls(p, pool(table=B, lens=B + 0x1000)))
    assert all(st == UNSUP for st in calls(p, pool(table=A + 4, lens=B, refs=B + 0x1000)))
    assert list(calls(p, p, n=-1))[:3] == [SHAPE] * 3
    assert list(calls(p, p, rows=None))[:3] == [NULL] * 3 and list(calls(p, p, rows=A + 1))[:3] == [ALIGN] * 3
    got = list(calls(p, p, word=None))
    assert got[0] == got[1] == got[3] == NULL
    got = list(calls(p, p, ws=None))
    assert got[0] == got[1] == got[3] == NULL
    need = lib.qbn_kv_pool_workspace(p, 2)
    assert need > 0 and list(calls(p, p, size=need - 1))[0] == SHAPE
    assert list(calls(p, p, c=cache(pages=9)))[1::2] == [SHAPE, SHAPE]
    assert list(calls(p, p, c=cache(page=32)))[1::2] == [SHAPE, SHAPE]
    assert lib.qbn_kv_free(p, p, 2, A, -1, 0, None) == SHAPE
    assert lib.qbn_kv_pool_workspace(None, 0) == -1 and lib.qbn_kv_pool_workspace(p, -1) == -1


def test_binding_checks():
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        qbn.KVCache("bf16", k, k)
    with pytest.raises(ValueError, match="unknown cache format"):
        qbn.KVCache("q4_0", k, k)
    with pytest.raises(ValueError, match="alike"):
        qbn.KVCache("bf16", k, k[:, :3])
    with pytest.raises(ValueError, match="unsupported cache shape"):
        qbn.KVCache("bf16", k[..., :8], k[..., :8])
    with pytest.raises(ValueError, match="no scales"):
        qbn.KVCache("bf16", k, k, k, k)
    with pytest.raises(ValueError, match="k_scales"):
        qbn.KVCache("mxfp8", k.to(torch.uint8), k.to(torch.uint8))
    with pytest.raises(TypeError):
        qbn.KVCache("mxfp8", k, k, torch.zeros(1, 4, 2, 2, 16, dtype=torch.uint8),
                    torch.zeros(1, 4, 2, 2, 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="device"):
        qbn.KVPool.empty(3, 4, 5, 16, device="cpu")
    with pytest.raises(TypeError):
        qbn.KVPool(torch.zeros(3, 4), torch.zeros(3), torch.zeros(5), 16)


def test_reference_pins():
    """The reference's element tables against torch's float8 types, its
    attention against a softmax written out for three tokens."""
    assert np.array_equal(R.FP8[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    assert np.array_equal(R.e8m0(np.arange(255)),
                          torch.arange(255, dtype=torch.uint8).view(torch.float8_e8m0fnu).double().numpy())
    assert R.FP4[7] == 6 and R.FP4[9] == -0.5 and np.signbit(R.FP4[8])
    x = np.array([[5.0, 2.5, 0.25, -1.75] + [0.0] * 28])
    code, scale = R.quantize("mxfp4", x)  # exponent 2 - 2 = 0: 5 -> 4, 2.5 -> 2, 0.25 -> 0, -1.75 -> -2 (ties to even)
    assert scale[0, 0] == 127 and list(code[0, :4]) == [6, 4, 0, 12]
    q, k, v = np.array([1.0, 0.0]), np.array([[0.0, 9], [1, 9], [2, 9]]), np.array([[1.0], [2.0], [4.0]])
    o, l, _, _, n = R.attention(q, k, v, 2, 0, 0, 1.0)
    e = np.exp([0.0, 1.0, 2.0])
    assert np.isclose(o[0], (e @ [1, 2, 4]) / e.sum()) and np.isclose(l, np.log(e.sum())) and n == 3
    o, l, _, _, n = R.attention(q, k, v, 2, 1, 1, 1.0)  # the last token and one sink
    assert np.isclose(o[0], (e[0] + 4 * e[2]) / (e[0] + e[2])) and n == 2
    assert R.attention(q, k, v, -1, 0, 0, 1.0)[1] == -np.inf
