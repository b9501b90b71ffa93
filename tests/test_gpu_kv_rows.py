"""GPU: which rows of q, k and v are whose. Rows that no sequence has (before
cu[0], from cu[seqs] on) and calls without cu, against the references of
test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
from gpu_util import DEV, say
from test_gpu_kv_attention import FORMATS, check, decode, fill, prefill, random_cache, vectors

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seqs,each", [(2, 1), (2, 40), (70, 1), (70, 40)])
def test_append_leaves_rows_of_no_sequence_out(fmt, seqs, each):
    """cu starts after row 0 and ends before the last row: the rows outside it are
    written nowhere, above all not over a sequence's earlier tokens."""
    rng = np.random.default_rng(seqs + each)
    ps, heads, dim, row, before, after = 16, 2, 64, 8, 9, 5
    news = [each] * seqs
    lens = [n + 30 for n in news]
    pages = sum(-(-n // ps) for n in lens)
    table = R.torch_table(lens, ps, row, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, None, junk=0x5A)
    want = [t.cpu() if t is not None else None for t in (c.k, c.v, c.k_scales, c.v_scales)]
    cu = before + np.concatenate([[0], np.cumsum(news)])
    x = [vectors(rng, int(cu[-1]) + after, heads, dim) for _ in range(2)]
    say("append", fmt, seqs, each)
    qbn.kv_append(c, x[0].to(DEV), x[1].to(DEV), table.to(DEV), ints(lens), ints(cu.tolist()))
    torch.cuda.synchronize()
    for which in (0, 1):
        code, scale = (None, None) if fmt == "bf16" else R.quantize(fmt, x[which].double().numpy())
        if fmt == "mxfp4":
            code = code[..., 0::2] | (code[..., 1::2] << 4)
        for b in range(seqs):
            for i in range(news[b]):
                pos, t = lens[b] - news[b] + i, int(cu[b]) + i
                page = int(table[b, pos // ps])
                want[which][0, page, :, pos % ps] = x[which][t] if code is None else torch.from_numpy(code[t])
                if code is not None:
                    want[which + 2][0, page, :, :, pos % ps] = torch.from_numpy(scale[t])
    for got, w, name in zip((c.k, c.v, c.k_scales, c.v_scales), want, ("k", "v", "k_scales", "v_scales")):
        if w is not None:
            assert torch.equal(got.cpu().view(torch.uint8), w.view(torch.uint8)), name


@pytest.mark.parametrize("fmt,dim", [("bf16", 64), ("mxfp8", 96), ("mxfp4", 256)])
@pytest.mark.parametrize("seqs", [1, 3, 64, 65, 130])
@pytest.mark.parametrize("before,after", [(0, 37), (3, 0), (70, 300), (0, 0)])
@pytest.mark.parametrize("wide", [False, True])
def test_prefill_rows_of_no_sequence(fmt, dim, seqs, before, after, wide):
    """Padding around the sequences' rows sees nothing: 0 and -inf, in the whole
    and in the split form, whatever out, lse and the workspace held."""
    rng = np.random.default_rng(seqs + before + after)
    ps, heads, group = 16, 1, 3
    lens = [int(n) for n in rng.integers(0, 90, seqs)]
    lens[0] = 77
    news = [int(rng.integers(0, min(n, 9) + 1)) for n in lens]
    pages = sum(-(-n // ps) for n in lens) + 1
    table = R.torch_table(lens, ps, 6, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    fill(c, table, lens, rng)
    cu = before + np.concatenate([[0], np.cumsum(news)])
    tokens = int(cu[-1]) + after
    if tokens == 0:
        return
    q = vectors(rng, tokens, heads * group, dim, gain=2.0)
    if wide:  # room for many pages: the split form
        table = torch.cat([table, torch.full((seqs, 400), -1, dtype=torch.int32)], 1)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    ws = torch.full((16 << 20,), 7.0, device=DEV)
    prefill(c, q, cu.tolist(), table, lens, out=out, lse=lse, workspace=ws)
    a, b = int(cu[0]), int(cu[-1])
    for rows in (slice(0, a), slice(b, tokens)):
        assert (out[rows] == 0).all() and (lse[rows] == -float("inf")).all()
    check(c, out[a:b], lse[a:b], q[a:b], table, lens, news, 0, 0)


@pytest.mark.parametrize("cu", [
    [0, 5, 3, 8], [0, 3, 5, 9], [-1, 3, 5, 8], [2, 1, 0, 8], [8, 8, 8, 0], [0, 2 ** 31 - 1, 4, 8], [0, -2 ** 31, 4, 8],
    [5, 3, 2, 1],
])
@pytest.mark.parametrize("seqs", [3, 67])
@pytest.mark.parametrize("wide", [False, True])
def test_prefill_rows_out_of_order_give_nan(cu, seqs, wide):
    """A cu that does not ascend, or leaves q: every output is NaN, none is left as it was."""
    rng = np.random.default_rng(seqs)
    ps, dim, tokens = 16, 64, 8
    cu = cu + [cu[-1]] * (seqs - 3)
    lens = [40] * seqs
    table = R.torch_table(lens, ps, 3, 3 * seqs, rng)
    c = random_cache("mxfp8", 3 * seqs, 1, ps, dim, rng)
    fill(c, table, lens, rng)
    if wide:
        table = torch.cat([table, torch.full((seqs, 400), -1, dtype=torch.int32)], 1)
    q = vectors(rng, tokens, 2, dim)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    prefill(c, q, cu, table, lens, out=out, lse=lse, workspace=torch.full((16 << 20,), 7.0, device=DEV))
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seqs,heads,group,dim", [(1, 1, 1, 64), (5, 2, 4, 128), (67, 1, 3, 96), (3, 1, 300, 64), (130, 2, 2, 256)])
@pytest.mark.parametrize("window,sinks,wide", [(0, 0, False), (0, 0, True), (50, 3, True)])
def test_prefill_of_one_token_each(fmt, seqs, heads, group, dim, window, sinks, wide):
    """Without cu every sequence has one new token, as in decode."""
    rng = np.random.default_rng(seqs + dim)
    ps = 32
    lens = [int(n) for n in rng.integers(0, 200, seqs)]
    lens[0], lens[-1] = 1, 190
    pages = sum(-(-n // ps) for n in lens) + 1
    table = R.torch_table(lens, ps, 200 // ps + 1, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    fill(c, table, lens, rng)
    if wide:
        table = torch.cat([table, torch.full((seqs, 300), -1, dtype=torch.int32)], 1)
    q = vectors(rng, seqs, heads * group, dim, gain=2.0)
    say("prefill, one each", fmt, dim, seqs, window)
    out, lse = qbn.kv_attention_prefill(c, q.to(DEV), None, table.to(DEV), ints(lens), window=window, sinks=sinks)
    torch.cuda.synchronize()
    check(c, out, lse, q, table, lens, [1] * seqs, window, sinks)
    # the same rows with cu written out
    out, lse = prefill(c, q, list(range(seqs + 1)), table, lens, window=window, sinks=sinks)
    check(c, out, lse, q, table, lens, [1] * seqs, window, sinks)


@pytest.mark.parametrize("seqs", [1000, 4097])
def test_thousands_of_sequences(seqs):
    """Lengths and row lists of many sequences: empty ones, long ones at the ends
    of a search's steps, decode and chunks, the same bits twice."""
    rng = np.random.default_rng(seqs)
    ps, dim, heads, group = 16, 64, 1, 2
    lens = [int(x) for x in rng.integers(0, 30, seqs)]
    for i, n in ((0, 0), (1, 900), (63, 500), (64, 0), (65, 1300), (seqs // 2, 2000), (seqs - 1, 1)):
        lens[i] = n
    news = [int(rng.integers(0, min(n, 3) + 1)) for n in lens]
    pages = sum(-(-n // ps) for n in lens) + 1
    table = R.torch_table(lens, ps, 2000 // ps + 1, pages, rng)
    c = random_cache("mxfp8", pages, heads, ps, dim, rng)
    fill(c, table, lens, rng)
    q = vectors(rng, seqs, heads * group, dim, gain=2.0)
    out, lse = decode(c, q, table, lens)
    check(c, out, lse, q, table, lens, [1] * seqs, 0, 0)
    again, lse2 = decode(c, q, table, lens)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    cu = [0] + np.cumsum(news).tolist()
    q = vectors(rng, cu[-1], heads * group, dim, gain=2.0)
    out, lse = prefill(c, q, cu, table, lens)
    check(c, out, lse, q, table, lens, news, 0, 0)


def test_calls_grow_with_the_sequences_not_with_their_square():
    """Eight times as many sequences of one short context: the time may grow by
    that factor and half of it again, not by its square."""
    def times(seqs):
        ps, dim, heads = 16, 64, 4
        c = qbn.KVCache.empty("mxfp8", 1, seqs, heads, ps, dim, device=DEV)
        for t in (c.k, c.v, c.k_scales, c.v_scales):
            t.fill_(100)
        table = torch.full((seqs, 64), -1, dtype=torch.int32, device=DEV)
        table[:, 0] = torch.arange(seqs, device=DEV)
        lens = torch.full((seqs,), 16, dtype=torch.int32, device=DEV)
        x = torch.ones(seqs, heads, dim, dtype=torch.bfloat16, device=DEV)
        cu = torch.arange(seqs + 1, dtype=torch.int32, device=DEV)
        calls = [lambda: qbn.kv_append(c, x, x, table, lens, cu), lambda: qbn.kv_attention_decode(c, x, table, lens),
                 lambda: qbn.kv_attention_prefill(c, x, cu, table, lens)]
        got = []
        for i, f in enumerate(calls):
            say("many", seqs, ("append", "decode", "prefill")[i])
            best = float("inf")
            for _ in range(5):
                a, b = torch.cuda.Event(True), torch.cuda.Event(True)
                a.record()
                f()
                b.record()
                b.synchronize()
                best = min(best, a.elapsed_time(b))
            say("%.3f ms" % best)
            got.append(best)
        return got

    few, many = times(8192), times(65536)
    for name, a, b in zip(("append", "decode", "prefill"), few, many):
        assert b <= 12 * a, "%s: %.3f ms for 8192 sequences, %.3f for 65536" % (name, a, b)


@pytest.mark.parametrize("fmt", FORMATS)
def test_empty_batches(fmt):
    """No sequences, or no rows: nothing is written, the outputs are empty."""
    c = random_cache(fmt, 2, 1, 16, 64, None, junk=0x5A)
    before = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]
    x = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    none, some = torch.zeros(0, 3, dtype=torch.int32, device=DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    say("empty", fmt)
    for table, lens, cu in ((none, ints([]), None), (none, ints([]), ints([0])), (some, ints([5, 0]), ints([0, 0, 0]))):
        qbn.kv_append(c, x, x, table, lens, cu)
        got = [qbn.kv_attention_prefill(c, q, cu, table, lens)]
        if cu is None:
            got.append(qbn.kv_attention_decode(c, q, table, lens))
        for out, lse in got:
            assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    torch.cuda.synchronize()
    for t, was in zip([t for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None], before):
        assert torch.equal(t.view(torch.uint8), was.view(torch.uint8))


def test_many_sequences_in_a_graph():
    """A step of more sequences than the waves scan, captured and replayed beside
    eager calls while lengths and rows change in place."""
    rng = np.random.default_rng(12)
    seqs, ps, dim, heads = 300, 16, 64, 2
    lens = rng.integers(1, 120, seqs)
    table = R.torch_table([int(n) + 8 for n in lens], ps, 64, 9 * seqs, rng).to(DEV)
    c = random_cache("mxfp4", 9 * seqs, heads, ps, dim, rng)
    fill(c, table.cpu(), [int(n) for n in lens], rng)
    k, v = (torch.zeros(2 * seqs, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros(2 * seqs, 4 * heads, dim, dtype=torch.bfloat16, device=DEV)
    n, cu = ints(lens.tolist()), ints((2 * np.arange(seqs + 1)).tolist())

    def step():
        qbn.kv_append(c, k, v, table, n, cu)
        return qbn.kv_attention_decode(c, q[:seqs], table, n) + qbn.kv_attention_prefill(c, q, cu, table, n)

    n.add_(2)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for rep in range(4):
        for t in (q, k, v):
            t.copy_(vectors(rng, *t.shape))
        n.add_(1)
        cu.copy_(ints(np.concatenate([[rep], np.sort(rng.integers(rep, 2 * seqs, seqs - 1)), [2 * seqs - rep]]).tolist()))
        torch.cuda.synchronize()
        say("graph replay", rep)
        g.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)]
        want = step()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        for x, y in zip(after, (c.k, c.v, c.k_scales, c.v_scales)):
            assert torch.equal(x, y)
    del g
