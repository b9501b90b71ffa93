"""The paged cache's call module without a GPU: it imports, and refuses, before
anything is enqueued, what the C ABI cannot see. No pointer is dereferenced:
every call below fails its checks or has nothing to do."""
import ctypes

import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
from bit_block_quantized_nibble_amd import kv

A = 0x10000


@pytest.fixture(scope="module")
def call():
    return kv._call()


def cache(heads=2, dim=64, format=16):
    return bytes(kv._CCache(format, heads, dim, 16, 1, 8, A, A, A, A))


def pool(**kw):
    f = dict(seqs=4, row=8, pages=8, page=16, table=A, lens=A + 0x1000, refs=A + 0x2000)
    f.update(kw)
    return bytes(kv._CPool(f["seqs"], f["row"], f["pages"], f["page"], 0, f["table"], f["lens"], f["refs"]))


BF, I32 = torch.bfloat16, torch.int32
K, T, L = torch.zeros(4, 2, 64, dtype=BF), torch.zeros(4, 8, dtype=I32), torch.zeros(4, dtype=I32)
CU = torch.zeros(5, dtype=I32)


# On a CPU tensor the device check comes last but before any call: "another
# device" says that everything before it passed.
@pytest.mark.parametrize("kw,error,words", [
    (dict(), ValueError, "another device"),
    (dict(k=K[:, :1]), ValueError, r"k must be \[tokens\]\[2\]\[64\]"),
    (dict(k=K[0]), ValueError, "k must be"),
    (dict(k=K.transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "last axis of k must be contiguous"),
    (dict(k=None), TypeError, "k must be a tensor"),
    (dict(cache=b"short"), TypeError, "not a handle"),
    (dict(cache=7), TypeError, "not a handle"),
    (dict(device="cuda"), TypeError, None),
])
def test_append_checks(call, kw, error, words):
    a = dict(cache=cache(), device=0, k=K, v=K, table=T, lens=L, cu=None, layer=0)
    a.update(kw)
    with pytest.raises(error, match=words):
        call.append(*a.values())


@pytest.mark.parametrize("kw,error,words", [
    (dict(v=K[:3]), ValueError, "alike"),
    (dict(v=K.float()), ValueError, "alike"),
    (dict(k=K.half(), v=K.half()), TypeError, "k dtype"),
    (dict(table=T.long()), TypeError, "table dtype"),
    (dict(table=T[0]), ValueError, r"table must be \[seqs\]\[row\]"),
    (dict(table=T.t().contiguous().t()), ValueError, "contiguous rows"),
    (dict(table=T[:3], lens=L[:3]), ValueError, "4 tokens for 3 sequences"),
    (dict(lens=L[:3]), ValueError, "lens has 3 entries; the call needs 4"),
    (dict(lens=L.long()), TypeError, "lens dtype torch.Long|lens dtype"),
    (dict(lens=torch.zeros(8, dtype=I32)[::2]), ValueError, "contiguous vector"),
    (dict(cu=CU[:4]), ValueError, "cu has 4 entries; the call needs 5"),
    (dict(cu=3), TypeError, "cu must be a tensor"),
])
def test_batch_checks(call, kw, error, words):
    """Device -1 is the CPU's: the checks behind the device's are reached."""
    a = dict(cache=cache(), device=-1, k=K, v=K, table=T, lens=L, cu=None, layer=0)
    a.update(kw)
    with pytest.raises(error, match=words):
        call.append(*a.values())


@pytest.mark.parametrize("kw,error,words", [
    (dict(q=K.float()), TypeError, "q dtype"),
    (dict(out=K[:3]), ValueError, "out must be contiguous"),
    (dict(out=K.float()), TypeError, "out dtype"),
    (dict(lse=torch.zeros(4, 3)), ValueError, "lse must be contiguous"),
    (dict(lse=torch.zeros(4, 2, dtype=torch.float64)), TypeError, "lse dtype"),
    (dict(workspace=torch.zeros(1), table=torch.zeros(4, 4096, dtype=I32)), ValueError, "workspace holds 4 bytes"),
    (dict(scale="x"), TypeError, None),
    (dict(window="x"), TypeError, None),
])
@pytest.mark.parametrize("decode", [True, False])
def test_attention_checks(call, decode, kw, error, words):
    a = dict(decode=decode, cache=cache(), device=-1, q=K, cu=None, table=T, lens=L, window=0, sinks=0, scale=0.1, layer=0,
             out=None, lse=None, workspace=None)
    a.update(kw)
    with pytest.raises(error, match=words):
        call.attention(*a.values())


def test_counts_of_arguments(call):
    for f in (call.append, call.attention, call.pool, call.pool_like, call.reserve, call.fork, call.release, call.compact):
        with pytest.raises(TypeError, match="wanted"):
            f()


@pytest.mark.parametrize("kw,error,words", [
    (dict(rows=L.long()), TypeError, "rows dtype"),
    (dict(tokens=L[:3]), ValueError, "tokens has 3 entries"),
    (dict(status=L), ValueError, "status has 4 entries; the call needs 1"),
    (dict(workspace=L), ValueError, "workspace holds 16 bytes"),
    (dict(device=0), ValueError, "another device"),
])
def test_reserve_checks(call, kw, error, words):
    a = dict(a=pool(), b=pool(), device=-1, rows=L, tokens=L, status=None, workspace=None)
    a.update(kw)
    with pytest.raises(error, match=words):
        call.reserve(*a.values())


def test_pool_checks(call):
    with pytest.raises(ValueError, match="device"):
        call.pool(T, L, L, 16)
    with pytest.raises(TypeError, match="table dtype"):
        call.pool(T.float(), L, L, 16)
    with pytest.raises(ValueError, match="contiguous"):
        call.pool(T.t(), L, L, 16)


def test_values_beyond_32_bits_are_refused_not_wrapped():
    lib = kv._kv()
    heads = ctypes.byref(kv._CCache(16, 4097, 64, 16, 1, 8, A, A, None, None))
    b = ctypes.byref(kv._CBatch(4, 4, 8, 8, A, A, None))
    assert lib.qbn_kv_append(heads, 0, b, A, 1 << 20, 64, A, 1 << 20, 64, 1, None) == 4  # more heads than a cache has
    assert qbn.kv_nbytes("bf16", 1, 8, 4096, 16, 64) > 0 and qbn.kv_nbytes("bf16", 1, 8, 4097, 16, 64) == -1
