"""GPU: turning vectors by their positions, alone and on the way into the paged
cache, against the formula with angles in extended precision."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
import step_ref as S
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def frequencies(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def ints(v):
    return torch.tensor(np.asarray(v).tolist(), dtype=torch.int32, device=DEV)


def vectors(rng, tokens, heads, dim, dt, gain=1.0):
    return torch.from_numpy((rng.standard_normal((tokens, heads, dim)) * gain).astype(np.float32)).to(DTYPES[dt])


def check(got, x, pos, freq, layout, factor=1.0, dt=None):
    want, tol = S.turn(x.double().numpy(), pos, freq, layout, factor)
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    g = got.cpu().double().numpy()
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), "%d of %d values off, first at %s: %r for %r +- %g" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], want[bad][0], tol[bad][0])
    rot = 2 * len(freq)
    assert torch.equal(got.cpu()[..., rot:], x[..., rot:].to(got.dtype))  # what does not turn stays


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [
    (1, 1, 16, 16), (1, 40, 128, 128), (3, 5, 96, 48), (17, 7, 80, 32), (2, 3, 64, 16), (5, 1, 192, 96), (4, 9, 256, 256),
    (33, 2, 48, 48), (1, 70, 1024, 1024), (2, 2, 1008, 992), (700, 3, 112, 64)])
def test_turns(layout, dt, tokens, heads, dim, rot):
    rng = np.random.default_rng(tokens + dim)
    x = vectors(rng, tokens, heads, dim, dt)
    pos = rng.integers(0, 200_000, tokens)
    f = frequencies(rot)
    say("rope", layout, dt, tokens, heads, dim, rot)
    check(qbn.rope(x.to(DEV), ints(pos), qbn.Rope(f, layout)), x, pos, f, layout)


def test_many_tokens():
    """More waves than the grid has: each takes several tokens."""
    rng = np.random.default_rng(5)
    x, pos, f = vectors(rng, 40_001, 2, 32, "bf16"), rng.integers(0, 1 << 20, 40_001), frequencies(32)
    say("rope many")
    check(qbn.rope(x.to(DEV), ints(pos), qbn.Rope(f)), x, pos, f, "half")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(layout):
    """Whole turns fall out exactly at any int32, with frequencies of several turns
    a position, of none, and negative ones."""
    pos = [0, 1, -1, 2**31 - 1, -2**31, 1_000_003, -77_777, 2**30]
    f = [1.0, 6.283185307179586, 7.5, 1e-9, 0.0, -0.25, 3.0, 1e-3]
    rng = np.random.default_rng(0)
    x = vectors(rng, len(pos), 3, 32, "f32")
    say("rope far", layout)
    check(qbn.rope(x.to(DEV), ints(pos), qbn.Rope(f, layout, 1.375)), x, pos, f, layout, 1.375)


def test_position_zero_changes_nothing():
    x = vectors(np.random.default_rng(1), 4, 3, 64, "bf16").to(DEV)
    say("rope zero")
    assert torch.equal(qbn.rope(x, ints([0] * 4), qbn.Rope(frequencies(64))), x)


@pytest.mark.parametrize("scaling,more", [("linear", {}), ("ntk", {}), ("bands", dict(original=4096)), ("yarn", dict(original=4096))])
def test_scalings(scaling, more):
    rng = np.random.default_rng(2)
    x, pos = vectors(rng, 9, 2, 64, "f32"), rng.integers(0, 100_000, 9)
    r = qbn.Rope.make(64, scaling=scaling, scale=8.0, layout="half", **more)
    say("rope", scaling)
    check(qbn.rope(x.to(DEV), ints(pos), r), x, pos, r.frequencies, "half", float(np.float32(r.factor)))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (96, 32), (192, 192)])
def test_views_and_in_place(layout, dt, dim, rot):
    """q of a fused projection turned in its place: the same bits as into a new
    tensor, and nothing beside it changes; transposed outputs."""
    rng = np.random.default_rng(dim)
    wide = vectors(rng, 37, 11, dim, dt).to(DEV)
    before = wide.clone()
    pos, r = ints(rng.integers(0, 9999, 37)), qbn.Rope(frequencies(rot), layout)
    q = wide[:, 2:9]
    say("rope views", layout, dt, dim)
    new = qbn.rope(q, pos, r)
    assert torch.equal(wide, before)
    heads_first = torch.empty(7, 37, dim, dtype=q.dtype, device=DEV).transpose(0, 1)
    assert qbn.rope(q, pos, r, out=heads_first) is not None and torch.equal(heads_first, new)
    assert qbn.rope(q, pos, r, out=q).data_ptr() == q.data_ptr()
    assert torch.equal(wide[:, 2:9], new)
    assert torch.equal(wide[:, :2], before[:, :2]) and torch.equal(wide[:, 9:], before[:, 9:])
    broadcast = before[:, :1].expand(-1, 6, -1)  # one head read six times
    assert torch.equal(qbn.rope(broadcast, pos, r), qbn.rope(broadcast.contiguous(), pos, r))


def test_infinities_and_nan_stay_in_their_pairs():
    x = torch.ones(1, 1, 64)
    x[0, 0, 3], x[0, 0, 50] = float("inf"), float("nan")
    say("rope nan")
    y = qbn.rope(x.to(DEV), ints([5]), qbn.Rope(frequencies(64))).cpu()
    bad = (~torch.isfinite(y[0, 0])).nonzero()[:, 0].tolist()
    assert bad == [3, 18, 35, 50]


def test_empty():
    r = qbn.Rope(frequencies(32))
    assert qbn.rope(torch.empty(0, 4, 32, device=DEV), ints([]), r).shape == (0, 4, 32)
    assert qbn.rope(torch.empty(3, 0, 32, device=DEV), ints([1, 2, 3]), r).shape == (3, 0, 32)


def test_refusals_on_the_device():
    r, x = qbn.Rope(frequencies(32)), torch.zeros(4, 2, 64, device=DEV)
    with pytest.raises(qbn.QbnError):  # it overlaps its source without being it
        qbn.rope(x[:3], ints([0] * 3), r, out=x[1:])
    with pytest.raises(qbn.QbnError):
        qbn.rope(x[:, :, :24], ints([0] * 4), r)  # dim no multiple of 16
    with pytest.raises(qbn.QbnError):
        qbn.rope(x[:, :, 2:34], ints([0] * 4), r)  # not 16-byte aligned
    with pytest.raises(qbn.QbnError):
        qbn.rope(x[:, :, :16], ints([0] * 4), r)  # rot beyond dim
    with pytest.raises(qbn.QbnError):  # two tokens in one place
        qbn.rope(x, ints([0] * 4), r, out=torch.empty(1, 2, 64, device=DEV).expand(4, -1, -1))
    with pytest.raises(ValueError, match="another device"):
        qbn.rope(x, torch.zeros(4, dtype=torch.int32), r)


# ---------------------------------------------------------------- on the way into the cache

FORMATS = ["bf16", "mxfp8", "mxfp4"]


def empty_cache(fmt, pages, heads, ps, dim, layers=1):
    c = qbn.KVCache.empty(fmt, layers, pages, heads, ps, dim)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        if t is not None:
            t.view(torch.uint8).fill_(0x5A)
    return c


def check_append(fmt, dt, layout, seqs, news, lens, heads, q_heads, dim, rot, ps=16, use_cu=True, layer=0, layers=1,
                 factor=1.0, in_place=False):
    rng = np.random.default_rng(sum(lens) + dim)
    tokens = sum(news)
    pages = sum(-(-n // ps) for n in lens) + 2
    table = R.torch_table(lens, ps, max(-(-n // ps) for n in lens) + 1, pages, rng)
    c = empty_cache(fmt, pages, heads, ps, dim, layers)
    want = [t.cpu().clone() if t is not None else None for t in (c.k, c.v, c.k_scales, c.v_scales)]
    x = vectors(rng, tokens, q_heads + 2 * heads, dim, dt)
    xd = x.to(DEV)
    q, k, v = xd.split([q_heads, heads, heads], 1)
    f = frequencies(rot)
    r = qbn.Rope(f, layout, factor)
    cu = np.concatenate([[0], np.cumsum(news)])
    say("append", fmt, dt, layout, seqs, dim, rot)
    got = qbn.kv_append_rope(c, q if q_heads else None, k, v, table.to(DEV), ints(lens), r, ints(cu) if use_cu else None,
                             layer=layer, out=q if in_place else None)
    torch.cuda.synchronize()
    pos = np.concatenate([np.arange(n - t, n) for n, t in zip(lens, news)]) if tokens else np.zeros(0)
    where = [(b, p) for b, (n, t) in enumerate(zip(lens, news)) for p in range(n - t, n)]
    if q_heads:
        assert got.dtype == torch.bfloat16
        want_q, tol = S.turn(x[:, :q_heads].double().numpy(), pos, f, layout, factor)
        tol = tol + 2.0 ** -8 * (np.abs(want_q) + tol)
        assert (np.abs(got.cpu().double().numpy() - want_q) <= tol).all()
    else:
        assert got is None
    if not in_place:
        assert torch.equal(xd.cpu(), x)
    kk, tol = S.turn(x[:, q_heads:q_heads + heads].double().numpy(), pos, f, layout, factor)
    vv = x[:, q_heads + heads:].double().numpy()
    for part, scale, y, t, name in ((c.k, c.k_scales, kk, tol, "k"), (c.v, c.v_scales, vv, np.zeros_like(vv), "v")):
        page = np.array([int(table[b, p // ps]) for b, p in where])
        slot = np.array([p % ps for b, p in where])
        part, scale = part.cpu(), None if scale is None else scale.cpu()
        stored = part[layer, page, :, slot]
        if fmt == "bf16":
            g = stored.double().numpy()
            assert (np.abs(g - y) <= t + 2.0 ** -8 * (np.abs(y) + t)).all(), name
        else:
            S.check_block(fmt, stored.numpy(), scale[layer, page, :, :, slot].numpy(), y, t, name)
        # nothing else changed
        i = 0 if name == "k" else 1
        want[i][layer, page, :, slot] = stored
        assert torch.equal(part.view(torch.uint8), want[i].view(torch.uint8)), name
        if scale is not None:
            want[i + 2][layer, page, :, :, slot] = scale[layer, page, :, :, slot]
            assert torch.equal(scale, want[i + 2]), name
    return c, got


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (96, 96), (96, 48), (128, 128), (128, 32), (192, 192), (192, 80),
                                     (256, 256), (256, 16)])
def test_append(fmt, layout, dt, dim, rot):
    check_append(fmt, dt, layout, 3, [1, 5, 2], [1, 37, 16], 3, 6, dim, rot)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seqs,use_cu", [(1, False), (5, False), (64, True), (65, True), (130, True)])
def test_append_sequences(fmt, seqs, use_cu):
    rng = np.random.default_rng(seqs)
    news = [1 if not use_cu else int(rng.integers(0, 4)) for _ in range(seqs)]
    news[0] = 1
    lens = [n + int(rng.integers(0, 60)) for n in news]
    lens = [max(1, n) for n in lens]
    check_append(fmt, "bf16", "half", seqs, news, lens, 2, 4, 64, 64, use_cu=use_cu, layer=1, layers=2, factor=1.25)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_without_queries(fmt):
    check_append(fmt, "bf16", "half", 2, [3, 1], [30, 9], 8, 0, 128, 128)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [192, 32])
def test_append_turns_queries_in_place(layout, rot):
    check_append("bf16", "bf16", layout, 2, [40, 1], [50, 9], 2, 5, 192, rot, in_place=True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_many_tokens(fmt):
    check_append(fmt, "bf16", "half", 2, [1500, 777], [1500, 2000], 3, 5, 96, 96, ps=64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_equals_rope_and_append(layout):
    """From binary32 sources the keys are those of rope followed by kv_append, bit for bit."""
    rng = np.random.default_rng(3)
    lens, news, ps, dim = [50, 20], [9, 20], 16, 96
    table = R.torch_table(lens, ps, 5, 8, rng).to(DEV)
    k, v = vectors(rng, 29, 2, dim, "f32").to(DEV), vectors(rng, 29, 2, dim, "f32").to(DEV)
    r = qbn.Rope(frequencies(dim), layout)
    cu, pos = ints([0, 9, 29]), ints(list(range(41, 50)) + list(range(20)))
    for fmt in FORMATS:
        a, b = empty_cache(fmt, 8, 2, ps, dim), empty_cache(fmt, 8, 2, ps, dim)
        say("append equals", fmt)
        qbn.kv_append_rope(a, None, k, v, table, ints(lens), r, cu)
        qbn.kv_append(b, qbn.rope(k, pos, r), v, table, ints(lens), cu)
        for s, t in ((a.k, b.k), (a.v, b.v), (a.k_scales, b.k_scales), (a.v_scales, b.v_scales)):
            assert s is None or torch.equal(s.view(torch.uint8), t.view(torch.uint8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seqs", [2, 70])
def test_append_rows_of_no_sequence(fmt, seqs):
    """Rows before cu[0] and from cu[seqs] on, more new tokens than a length has, bad
    pages and rows that are too short: nothing is stored, queries without a position are
    copied, the others turned."""
    rng = np.random.default_rng(seqs)
    dim, ps, pages = 64, 16, seqs + 4
    lens = [10] * seqs
    lens[1] = 1  # of two new tokens: the first has position -1
    table = torch.arange(seqs, dtype=torch.int32)[:, None].clone()
    table[0, 0] = pages  # no page of the cache
    cu = (3 + np.arange(seqs + 1) * 2).tolist()
    tokens = cu[-1] + 5
    x = vectors(rng, tokens, 4, dim, "bf16").to(DEV)
    c = empty_cache(fmt, pages, 1, ps, dim)
    before = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]
    r = qbn.Rope(frequencies(dim))
    say("append rows", fmt, seqs)
    q = qbn.kv_append_rope(c, x[:, :2], x[:, 2:3], x[:, 3:], table.to(DEV), ints(lens), r, ints(cu))
    torch.cuda.synchronize()
    assert torch.equal(q[:3], x[:3, :2]) and torch.equal(q[cu[-1]:], x[cu[-1]:, :2])
    assert torch.equal(q[cu[1]], x[cu[1], :2])  # position -1
    pos = np.array([0, 8 + 1])
    check(q[[cu[1] + 1, cu[0] + 1]], x[[cu[1] + 1, cu[0] + 1], :2].cpu(), pos, frequencies(dim), "half")
    changed = torch.zeros(1, pages, 1, ps, 1, dtype=torch.bool, device=DEV)
    changed[0, 1, 0, 0] = True
    changed[0, 2:seqs, 0, 8:10] = True
    for t, b in zip((c.k, c.v), before):
        same = (t.view(torch.uint8) == b.view(torch.uint8))
        assert same[~changed.expand_as(same)].all()
    # a table without columns: queries are turned, nothing is stored
    c2 = empty_cache(fmt, pages, 1, ps, dim)
    q2 = qbn.kv_append_rope(c2, x[:, :2], x[:, 2:3], x[:, 3:], table.to(DEV)[:, :0], ints(lens), r, ints(cu))
    assert torch.equal(q2, q)
    assert (c2.k.view(torch.uint8) == 0x5A).all() and (c2.v.view(torch.uint8) == 0x5A).all()


def test_append_refusals():
    rng = np.random.default_rng(0)
    c = empty_cache("bf16", 4, 2, 16, 64)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), ints([1])
    x = vectors(rng, 1, 8, 64, "bf16").to(DEV)
    q, k, v = x.split([4, 2, 2], 1)
    r = qbn.Rope(frequencies(64))
    with pytest.raises(ValueError, match="None"):
        qbn.kv_append_rope(c, None, k, v, table, lens, r, out=q)
    with pytest.raises(TypeError, match="out dtype"):
        qbn.kv_append_rope(c, q, k, v, table, lens, r, out=q.float())
    with pytest.raises(ValueError, match="alike"):
        qbn.kv_append_rope(c, q.float(), k, v, table, lens, r)
    with pytest.raises(qbn.QbnError):
        qbn.kv_append_rope(c, q, k, v, table, lens, qbn.Rope(frequencies(128)))  # rot beyond head_dim
    with pytest.raises(qbn.QbnError):
        qbn.kv_append_rope(c, q, k, v, table, lens, r, out=x[:, 2:6])  # over q and k
    with pytest.raises(qbn.QbnError):
        qbn.kv_append_rope(c, q, k, v, table, lens, r, layer=1)
    with pytest.raises(ValueError, match="another device"):
        qbn.kv_append_rope(c, q, k, v, table, lens, qbn.Rope(frequencies(64), device="cpu"))


def test_graph_replays():
    """Captured once, replayed on new contents: as the eager call."""
    rng = np.random.default_rng(9)
    lens, table = ints([5, 40]), torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32, device=DEV)
    x = vectors(rng, 2, 8, 64, "bf16").to(DEV)
    r = qbn.Rope(frequencies(64))
    a, b = empty_cache("mxfp8", 6, 2, 16, 64), empty_cache("mxfp8", 6, 2, 16, 64)
    q, k, v = x.split([4, 2, 2], 1)
    out = torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    pos = ints([4, 39])
    turned = torch.empty_like(out)
    say("graph")
    for c in (a, b):  # once before the capture, into both
        qbn.kv_append_rope(c, q, k, v, table, lens, r, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qbn.kv_append_rope(a, q, k, v, table, lens, r, out=out)
        qbn.rope(q, pos, r, out=turned)
    for i in range(3):
        x.copy_(vectors(rng, 2, 8, 64, "bf16"))
        lens.add_(1)
        pos.add_(1)
        g.replay()
        torch.cuda.synchronize()
        want = qbn.kv_append_rope(b, q, k, v, table, lens, r)
        assert torch.equal(out, want) and torch.equal(turned, want)
    # what the replays stored, the eager calls stored too
    for t, u in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(t, u)
