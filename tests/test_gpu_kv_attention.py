"""GPU: the paged key-value cache's append and attention kernels against plain
binary64 references (kv_ref.py). Appends are bit-exact; attention is held to
a bound that counts its roundings (kv_ref.attention_tolerance)."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

FORMATS = ("bf16", "mxfp8", "mxfp4")


def random_cache(fmt, pages, heads, ps, dim, rng, layers=1, junk=0xFF):
    """A cache whose unwritten parts hold junk (NaN patterns with 0xFF)."""
    c = qbn.KVCache.empty(fmt, layers, pages, heads, ps, dim, device=DEV)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        if t is not None:
            t.view(torch.uint8).fill_(junk)
    return c


def vectors(rng, *shape, dtype=torch.bfloat16, gain=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * gain).astype(np.float32)).to(dtype)


def fill(cache, table, lens, rng, layer=0, gain=1.0):
    """Append every token of every sequence; the K and V of each, as appended."""
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k = vectors(rng, cu[-1], cache.heads, cache.head_dim, gain=gain)
    v = vectors(rng, cu[-1], cache.heads, cache.head_dim)
    say("append", cache.format, list(lens))
    qbn.kv_append(cache, k.to(DEV), v.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                  torch.from_numpy(cu).to(DEV), layer=layer)
    torch.cuda.synchronize()
    return k, v


def held(cache, layer=0):
    s = (None, None) if cache.format == "bf16" else (cache.k_scales[layer].cpu(), cache.v_scales[layer].cpu())
    return (R.decode(cache.format, cache.k[layer].cpu(), s[0]), R.decode(cache.format, cache.v[layer].cpu(), s[1]))


def check(cache, out, lse, q, table, lens, news, window, sinks, scale=None, layer=0, rows=None):
    scale = cache.head_dim ** -0.5 if scale is None else scale
    with np.errstate(all="ignore"):
        k, v = held(cache, layer)
    out, lse, qd = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    group = q.shape[1] // cache.heads
    at, worst = 0, 0.0
    for b, (n, t) in enumerate(zip(lens, news)):
        for h in range(cache.heads):
            kk, vv = R.rows_of(k, table[b].tolist(), n, h), R.rows_of(v, table[b].tolist(), n, h)
            for i in range(t):
                if rows is not None and i not in rows:
                    continue
                for g in range(group):
                    o, l, w, reach, count = R.attention(qd[at + i, h * group + g], kk, vv, n - t + i, window, sinks, scale)
                    to, tl = R.attention_tolerance(cache.head_dim, o, w, l, reach, count)
                    got, gl = out[at + i, h * group + g], lse[at + i, h * group + g]
                    where = "sequence %d token %d head %d" % (b, i, h * group + g)
                    if count == 0:
                        assert (got == 0).all() and gl == -np.inf, where
                        continue
                    err = np.abs(got - o)
                    assert (err <= to).all(), "%s: off by %g of the bound" % (where, np.nanmax(err / to))
                    assert abs(gl - l) <= tl, "%s: lse %r, wanted %r" % (where, gl, l)
                    worst = max(worst, float((err / to).max()))
        at += t
    return worst


def decode(cache, q, table, lens, **kw):
    say("decode", cache.format, cache.head_dim, cache.page_size, tuple(q.shape), list(lens), kw)
    out, lse = qbn.kv_attention_decode(cache, q.to(DEV), table.to(DEV),
                                       torch.tensor(lens, dtype=torch.int32, device=DEV), **kw)
    torch.cuda.synchronize()
    return out, lse


def prefill(cache, q, cu, table, lens, **kw):
    say("prefill", cache.format, cache.head_dim, cache.page_size, tuple(q.shape), list(lens), list(cu), kw)
    out, lse = qbn.kv_attention_prefill(cache, q.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), table.to(DEV),
                                        torch.tensor(lens, dtype=torch.int32, device=DEV), **kw)
    torch.cuda.synchronize()
    return out, lse


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,dim,ps", [(1, 64, 16), (3, 96, 32), (8, 128, 64), (2, 192, 128), (5, 256, 256)])
def test_append_is_exact(fmt, dtype, heads, dim, ps):
    rng = np.random.default_rng(heads * dim + ps)
    lens, news = [ps + 3, 1, 2 * ps, 5], [ps, 1, 7, 5]
    width, layers, layer = 4, 2, 1
    table = R.torch_table(lens, ps, width, 12, rng)
    c = random_cache(fmt, 12, heads, ps, dim, rng, layers=layers, junk=0x5A)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    wide = vectors(rng, cu[-1], 2 * heads + 1, dim, dtype=torch.float32)
    # blocks of zeros, of -0, of tiny and of huge values, and ties of both element grids
    wide[0, 0, :32] = 0.0
    wide[1, 0, :32] = -0.0
    wide[2, 0, :32] *= 2.0 ** -120
    wide[3, 0, :32] *= 2.0 ** 100
    wide[4, 0, :32] = torch.arange(32) * 0.25 - 4.0
    wide[5, 0, :32] = torch.arange(32) * 0.03125 + 1.0
    wide = wide.to(dtype)
    k, v = wide[:, :heads], wide[:, heads + 1:]  # views of one projection
    before = [t.clone() if t is not None else None for t in (c.k, c.v, c.k_scales, c.v_scales)]
    say("append", fmt, dtype, heads, dim, ps)
    dw = wide.to(DEV)
    qbn.kv_append(c, dw[:, :heads], dw[:, heads + 1:], table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                  torch.from_numpy(cu).to(DEV), layer=layer)
    torch.cuda.synchronize()
    want = [t.cpu() if t is not None else None for t in before]
    for which, x in ((0, k), (1, v)):
        for b in range(len(lens)):
            for i in range(news[b]):
                pos = lens[b] - news[b] + i
                page, slot = int(table[b, pos // ps]), pos % ps
                row = x[cu[b] + i]
                if fmt == "bf16":
                    want[which][layer, page, :, slot] = row.to(torch.bfloat16)
                    continue
                code, scale = R.quantize(fmt, row.double().numpy())
                if fmt == "mxfp4":
                    code = code[..., 0::2] | (code[..., 1::2] << 4)
                want[which][layer, page, :, slot] = torch.from_numpy(code)
                want[which + 2][layer, page, :, :, slot] = torch.from_numpy(scale)
    for got, w, name in zip((c.k, c.v, c.k_scales, c.v_scales), want, ("k", "v", "k_scales", "v_scales")):
        if w is not None:
            assert torch.equal(got.cpu().view(torch.uint8), w.view(torch.uint8)), name


def test_append_one_token_each_and_strays():
    """cu = None; tokens without a page, before position 0 or beyond the row are dropped."""
    rng = np.random.default_rng(3)
    ps, c = 16, random_cache("mxfp8", 6, 2, 16, 64, None, junk=0)
    table = torch.tensor([[0, 1], [2, -1], [9, 3], [4, 5], [-7, 5]], dtype=torch.int32)
    lens = [18, 17, 3, 33, 0]  # page 1 slot 1; no page; page 9 of 6; beyond the row; before 0
    k, v = vectors(rng, 5, 2, 64), vectors(rng, 5, 2, 64)
    say("append strays")
    qbn.kv_append(c, k.to(DEV), v.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    want = torch.zeros_like(c.k.cpu())
    want[0, 1, :, 1] = torch.from_numpy(R.quantize("mxfp8", k[0].double().numpy())[0])
    assert torch.equal(c.k.cpu(), want)
    assert int((c.v_scales != 0).sum()) == 4


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("ps,heads,group", [(16, 2, 4), (64, 1, 7), (256, 3, 1)])
def test_decode(fmt, dim, ps, heads, group):
    rng = np.random.default_rng(dim + ps)
    lens = [1, 0, 31, 33, 128, 129, 300, 2 * ps - 1]
    width = max(lens) // ps + 3
    pages = sum(-(-n // ps) for n in lens) + 3
    table = R.torch_table(lens, ps, width, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    fill(c, table, lens, rng)
    q = vectors(rng, len(lens), heads * group, dim, gain=2.0)
    out, lse = decode(c, q, table, lens)
    check(c, out, lse, q, table, lens, [1] * len(lens), 0, 0)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (40, 0), (100, 4), (129, 33), (400, 130), (5000, 3)])
@pytest.mark.parametrize("fmt,ps", [("mxfp4", 16), ("bf16", 128)])
def test_decode_window_and_sinks(fmt, ps, window, sinks):
    rng = np.random.default_rng(window + sinks)
    lens, heads, group, dim = [2, 100, 777, 1500, 128], 2, 3, 64
    pages = sum(-(-n // ps) for n in lens)
    table = R.torch_table(lens, ps, 1500 // ps + 2, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    fill(c, table, lens, rng)
    # what slid out of the window may be gone or hold anything
    if fmt == "bf16":
        for b, n in enumerate(lens):
            for t in range(n):
                if sinks <= t < n - window:
                    c.k[0, int(table[b, t // ps]), :, t % ps] = float("nan")
                    c.v[0, int(table[b, t // ps]), :, t % ps] = float("inf")
    else:
        for b, n in enumerate(lens):
            for j in range(width := table.shape[1]):
                if sinks <= j * ps and (j + 1) * ps <= n - window:
                    table[b, j] = -1
    q = vectors(rng, len(lens), heads * group, dim, gain=2.0)
    out, lse = decode(c, q, table, lens, window=window, sinks=sinks)
    check(c, out, lse, q, table, lens, [1] * len(lens), window, sinks)


@pytest.mark.parametrize("group", [16, 17, 40])
def test_decode_many_query_heads(group):
    rng = np.random.default_rng(group)
    lens, ps = [700, 5], 32
    table = R.torch_table(lens, ps, 24, 30, rng)
    c = random_cache("mxfp8", 30, 1, ps, 128, rng)
    fill(c, table, lens, rng)
    q = vectors(rng, 2, group, 128)
    out, lse = decode(c, q, table, lens)
    check(c, out, lse, q, table, lens, [1, 1], 0, 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_long_split_and_joined(fmt):
    """Lengths far apart, so that the pieces of a sequence lie in many workgroups; the same bits twice."""
    rng = np.random.default_rng(17)
    lens, ps, heads, group, dim = [9000, 3, 0, 1, 4096, 260], 64, 2, 4, 128
    pages = sum(-(-n // ps) for n in lens)
    table = R.torch_table(lens, ps, 150, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    fill(c, table, lens, rng, gain=1.5)
    q = vectors(rng, len(lens), heads * group, dim, gain=2.0)
    out, lse = decode(c, q, table, lens)
    check(c, out, lse, q, table, lens, [1] * len(lens), 0, 0)
    again, lse2 = decode(c, q, table, lens)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_decode_strided_query_scale_and_layer():
    rng = np.random.default_rng(5)
    lens, ps, dim = [90, 41], 32, 64
    table = R.torch_table(lens, ps, 4, 8, rng)
    c = random_cache("mxfp4", 8, 2, ps, dim, rng, layers=3)
    fill(c, table, lens, rng, layer=2)
    wide = vectors(rng, 2, 10, 2 * dim).to(DEV)
    q = wide[:, 1:7, dim:]
    wide_table = torch.cat([table, torch.full((2, 5), 77, dtype=torch.int32)], 1).to(DEV)[:, :4]
    say("decode strided")
    out, lse = qbn.kv_attention_decode(c, q, wide_table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale=-0.3,
                                       layer=2)
    torch.cuda.synchronize()
    check(c, out, lse, q, table, lens, [1, 1], 0, 0, scale=float(np.float32(-0.3)), layer=2)


def test_decode_bad_pages_and_lengths_give_nan():
    """Entries that are no pages, lengths beyond the row or negative: NaN for
    that sequence, the others untouched."""
    rng = np.random.default_rng(6)
    lens, ps, dim = [90, 90, 90, 90, 90], 16, 64
    good = R.torch_table(lens, ps, 6, 30, rng)
    c = random_cache("bf16", 30, 1, ps, dim, rng)
    fill(c, good, lens, rng)
    q = vectors(rng, 5, 2, dim)
    for reach in (96, 10 ** 6):  # one workgroup a pair, and the split form (a wide row)
        table = good.clone()
        if reach > 96:
            table = torch.cat([table, torch.full((5, 94), -1, dtype=torch.int32)], 1)
        table[1, 2], table[2, 0] = 30, -1
        odd = [90, 90, 90, 16 * table.shape[1] + 1, -4]
        out, lse = decode(c, q, table, odd)
        assert torch.isnan(out[1:]).all() and torch.isnan(lse[1:]).all()
        check(c, out[:1], lse[:1], q[:1], good, [90], [1], 0, 0)


def test_decode_special_values():
    """Visible infinities and NaN act as in the formula; scores that overflow to -inf everywhere give 0."""
    rng = np.random.default_rng(8)
    ps, dim = 16, 64
    c = random_cache("bf16", 2, 1, ps, dim, rng)
    table, lens = torch.tensor([[1, 0]], dtype=torch.int32), [20]
    fill(c, table, lens, rng)
    q = vectors(rng, 1, 1, dim)
    c.v[0, 1, 0, 3, 5] = float("inf")
    c.v[0, 1, 0, 4, 6] = float("nan")
    out, lse = decode(c, q, table, lens)
    o = out[0, 0].float().cpu()
    assert o[5] == float("inf") and torch.isnan(o[6]) and torch.isfinite(o[[0, 4, 7, 63]]).all()
    c.k[0, 0, 0, 2] = float("nan")
    out, lse = decode(c, q, table, lens)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


# ------------------------------------------------------------------ prefill

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("ps,heads,group", [(16, 1, 4), (64, 2, 3), (256, 1, 1)])
def test_prefill(fmt, dim, ps, heads, group):
    rng = np.random.default_rng(dim + ps)
    lens, news = [1, 63, 200, 70, 0, 65], [1, 63, 40, 1, 0, 65]
    pages = sum(-(-n // ps) for n in lens) + 2
    table = R.torch_table(lens, ps, 200 // ps + 2, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    fill(c, table, lens, rng)
    cu = [0] + np.cumsum(news).tolist()
    q = vectors(rng, cu[-1], heads * group, dim, gain=2.0)
    out, lse = prefill(c, q, cu, table, lens)
    check(c, out, lse, q, table, lens, news, 0, 0)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (17, 0), (64, 4), (100, 70), (250, 1), (4000, 9)])
@pytest.mark.parametrize("fmt,ps", [("mxfp4", 32), ("bf16", 16)])
def test_prefill_window_and_sinks(fmt, ps, window, sinks):
    rng = np.random.default_rng(window + sinks)
    lens, news, heads, group, dim = [300, 555], [300, 33], 1, 2, 64
    pages = sum(-(-n // ps) for n in lens)
    table = R.torch_table(lens, ps, 555 // ps + 1, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    fill(c, table, lens, rng)
    cu = [0] + np.cumsum(news).tolist()
    q = vectors(rng, cu[-1], heads * group, dim, gain=2.0)
    out, lse = prefill(c, q, cu, table, lens, window=window, sinks=sinks)
    check(c, out, lse, q, table, lens, news, window, sinks)


def test_prefill_more_new_tokens_than_length_and_unused_rows():
    """Queries before position 0 see nothing; every format of cu's rows is covered."""
    rng = np.random.default_rng(9)
    ps, dim = 16, 128
    lens, news = [5, 0, 40], [9, 3, 8]
    table = R.torch_table(lens, ps, 3, 6, rng)
    c = random_cache("mxfp8", 6, 2, ps, dim, rng)
    fill(c, table, lens, rng)
    cu = [0] + np.cumsum(news).tolist()
    q = vectors(rng, cu[-1], 4, dim)
    out, lse = prefill(c, q, cu, table, lens)
    check(c, out, lse, q, table, lens, news, 0, 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_prefill_long_split_and_joined(fmt):
    rng = np.random.default_rng(21)
    lens, news, ps, dim = [3000, 50], [5, 2], 64, 128
    pages = sum(-(-n // ps) for n in lens)
    table = R.torch_table(lens, ps, 50, pages, rng)
    c = random_cache(fmt, pages, 2, ps, dim, rng)
    fill(c, table, lens, rng)
    q = vectors(rng, 7, 8, dim, gain=2.0)
    out, lse = prefill(c, q, [0, 5, 7], table, lens)
    check(c, out, lse, q, table, lens, news, 0, 0)
    again, lse2 = prefill(c, q, [0, 5, 7], table, lens)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_prefill_many_rows_sampled():
    """Several row tiles of a long chunk, sampled rows; decode of the last token agrees."""
    rng = np.random.default_rng(22)
    lens, news, ps, dim = [1500], [1100], 128, 128
    table = R.torch_table(lens, ps, 13, 12, rng)
    c = random_cache("mxfp4", 12, 2, ps, dim, rng)
    fill(c, table, lens, rng)
    q = vectors(rng, 1100, 6, dim, gain=2.0)
    out, lse = prefill(c, q, [0, 1100], table, lens, window=333, sinks=5)
    check(c, out, lse, q, table, lens, news, 333, 5, rows={0, 1, 41, 42, 43, 64, 500, 777, 1098, 1099})
    o1, l1 = decode(c, q[-1:], table, lens, window=333, sinks=5)
    assert (l1 - lse[-1:]).abs().max() < 1e-4
    assert (o1.float() - out[-1:].float()).abs().max() < 2.0 ** -6


@pytest.mark.parametrize("few", [True, False])
def test_prefill_infinities_in_masked_tokens(few):
    """An infinity or NaN of V reaches exactly the rows that see its token."""
    rng = np.random.default_rng(23)
    n, ps, dim = 1600, 16, 64
    t = 20 if few else 1600  # few rows: the split form
    table = R.torch_table([n], ps, 100, 100, rng)
    c = random_cache("bf16", 100, 1, ps, dim, rng)
    fill(c, table, [n], rng)
    q = vectors(rng, t, 1, dim)
    clean, lse0 = prefill(c, q, [0, t], table, [n], window=30, sinks=2)
    odd = {0: (3, float("inf")), 1: (3, float("-inf")), n - 5: (7, float("nan")), n - 12: (9, float("-inf")),
           n - 300: (11, float("inf")), n - 290: (12, float("nan"))}
    for tok, (d, x) in odd.items():
        c.v[0, int(table[0, tok // ps]), 0, tok % ps, d] = x
    out, lse = prefill(c, q, [0, t], table, [n], window=30, sinks=2)
    assert torch.equal(lse, lse0)
    got, was = out[:, 0].float().cpu().numpy(), clean[:, 0].float().cpu().numpy()
    want = was.copy()
    for i in range(t):
        pos = n - t + i
        for tok, (d, x) in odd.items():
            if tok <= pos and (tok > pos - 30 or tok < 2):
                with np.errstate(invalid="ignore"):
                    want[i, d] += x
    special = ~np.isfinite(want)
    assert special.any() and (np.isnan(want) == np.isnan(got)).all()
    assert (got[special & ~np.isnan(want)] == want[special & ~np.isnan(want)]).all()
    # the finite outputs are those of a V with 0 in the odd places, to the tolerance of a bf16 output
    fine = ~special
    fine[:, [d for d, _ in odd.values()]] = False
    assert (got[fine] == was[fine]).all()


def test_prefill_bad_pages_give_nan():
    rng = np.random.default_rng(24)
    lens, ps, dim = [80, 80, 80], 16, 64
    good = R.torch_table(lens, ps, 5, 15, rng)
    c = random_cache("mxfp8", 15, 1, ps, dim, rng)
    fill(c, good, lens, rng)
    q = vectors(rng, 30, 2, dim)
    table = good.clone()
    table[1, 1] = 15
    out, lse = prefill(c, q, [0, 10, 20, 30], table, [80, 80, 81])
    assert torch.isnan(out[10:]).all() and torch.isnan(lse[10:]).all()
    check(c, out[:10], lse[:10], q[:10], good, [80], [10], 0, 0)


# ------------------------------------------------------------------ together

def test_steps_in_a_graph_and_on_another_stream():
    """Append and attend, captured once and replayed while the inputs change in
    place, with eager steps between; then on a side stream. Bit-identical."""
    rng = np.random.default_rng(30)
    ps, dim, lens = 16, 128, [400, 77, 16]
    table = R.torch_table([n + 40 for n in lens], ps, 64, 64, rng).to(DEV)
    c = random_cache("mxfp4", 64, 2, ps, dim, rng)
    fill(c, table.cpu(), lens, rng)
    q, k, v = (torch.zeros(3, h, dim, dtype=torch.bfloat16, device=DEV) for h in (8, 2, 2))
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)

    def step():
        n.add_(1)
        qbn.kv_append(c, k, v, table, n)
        a = qbn.kv_attention_decode(c, q, table, n, window=300, sinks=4)
        b = qbn.kv_attention_prefill(c, q, cu, table, n, window=300, sinks=4)
        return a + b

    step()
    n.sub_(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    side = torch.cuda.Stream()
    for rep in range(4):
        for t in (q, k, v):
            t.copy_(vectors(rng, *t.shape))
        torch.cuda.synchronize()
        say("graph replay", rep)
        g.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)]
        n.sub_(1)
        torch.cuda.synchronize()
        if rep % 2:
            with torch.cuda.stream(side):
                want = step()
        else:
            want = step()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        for x, y in zip(after, (c.k, c.v, c.k_scales, c.v_scales)):
            assert torch.equal(x, y)
    del g


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    fmt, ps = FORMATS[rng.integers(3)], int(2 ** rng.integers(4, 9))
    dim, heads, group = int(rng.choice([64, 96, 128, 192, 256])), int(rng.integers(1, 4)), int(rng.integers(1, 10))
    lens = [int(x) for x in rng.integers(0, 500, rng.integers(1, 6))]
    news = [int(rng.integers(0, min(n, 20) + 1)) for n in lens]
    window = int(rng.choice([0, rng.integers(1, 300)]))
    sinks = int(rng.integers(0, 40))
    pages = sum(-(-n // ps) for n in lens) + 1
    table = R.torch_table(lens, ps, 500 // ps + int(rng.integers(1, 40)), pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    if sum(lens):
        fill(c, table, lens, rng)
    q = vectors(rng, len(lens), heads * group, dim)
    out, lse = decode(c, q, table, lens, window=window, sinks=sinks)
    check(c, out, lse, q, table, lens, [1] * len(lens), window, sinks)
    if sum(news):
        cu = [0] + np.cumsum(news).tolist()
        q = vectors(rng, cu[-1], heads * group, dim)
        out, lse = prefill(c, q, cu, table, lens, window=window, sinks=sinks)
        check(c, out, lse, q, table, lens, news, window, sinks)
