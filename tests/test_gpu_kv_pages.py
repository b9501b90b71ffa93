"""GPU: the paged cache's bookkeeping (reserve, fork, free, compact) against a
one-page-at-a-time reference, tables and payload bytes exactly."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), dtype=torch.int32, device=DEV)


def make(rng, fmt="mxfp4", layers=2, pages=40, heads=2, ps=16, dim=64, seqs=6, row=8, lens=(40, 16, 3, 0, 64, 0)):
    c = qbn.KVCache.empty(fmt, layers, pages, heads, ps, dim, device=DEV)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        if t is not None:
            b = t.view(torch.uint8)
            b.copy_(torch.from_numpy(rng.integers(0, 256, tuple(b.shape), dtype=np.uint8)))
    lens = list(lens) + [0] * (seqs - len(lens))
    table = R.torch_table(lens, ps, row, pages, rng)
    refs = np.zeros(pages, np.int32)
    for p in table.numpy().ravel():
        if p >= 0:
            refs[p] += 1
    pool = qbn.KVPool(table.to(DEV), ints(lens), ints(refs), ps)
    return c, pool, R.RefPool(table.numpy(), np.array(lens, np.int32), refs, ps)


def payload(c):
    return [t.cpu().view(torch.uint8).clone() for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]


def same(pool, ref):
    torch.cuda.synchronize()
    assert np.array_equal(pool.lens.cpu().numpy(), ref.lens)
    assert np.array_equal(pool.refs.cpu().numpy(), ref.refs)
    assert np.array_equal(pool.table.cpu().numpy(), ref.table)


def same_payload(c, before, moves):
    for t in before:
        for s, d in moves:
            t[:, d] = t[:, s]
    for got, want in zip(payload(c), before):
        assert torch.equal(got, want)


@pytest.mark.parametrize("fmt,page", [("bf16", 16), ("mxfp8", 64), ("mxfp4", 256)])
@pytest.mark.parametrize("separate", [False, True])
def test_a_turn(fmt, page, separate):
    rng = np.random.default_rng(page)
    lens = [int(x) for x in rng.integers(0, 5 * page, 9)] + [3 * page, page // 2]
    c, pool, ref = make(rng, fmt, layers=3, pages=200, ps=page, dim=96, seqs=20, row=12, lens=lens)
    before = payload(c)
    old = (pool.table.clone(), pool.lens.clone(), pool.refs.clone())
    for t in range(4):
        stay = [b for b in range(20) if ref.lens[b] > 0]
        gone = list(rng.choice(stay, max(1, len(stay) // 4), replace=False)) + [gone_twice := int(stay[0]), gone_twice, 99, -1]
        say("free", fmt, page, separate, t)
        after = qbn.KVPool.like(pool) if separate else pool
        qbn.kv_free(pool, ints(gone), out=after)
        ref.release(gone)
        same(after, ref)
        if separate and t == 0:
            for x, y in zip(old, (pool.table, pool.lens, pool.refs)):
                assert torch.equal(x, y)
        stay = [b for b in range(20) if ref.lens[b] > 0]
        empty = [b for b in range(20) if ref.lens[b] == 0]
        kids = empty[:min(3, len(empty))]
        parents = [int(x) for x in rng.choice(stay, len(kids))]
        ref.moves = []
        say("fork")
        nxt = qbn.KVPool.like(pool) if separate else pool
        st = qbn.kv_fork(c, after, ints(parents), ints(kids), out=nxt)
        assert ref.fork(parents, kids) == -1 and int(st) == -1
        same(nxt, ref)
        same_payload(c, before, ref.moves)
        rows = [b for b in range(20) if ref.lens[b] > 0]
        rng.shuffle(rows)
        room = [min(int(x), 12 * page - int(ref.lens[b])) for x, b in zip(rng.integers(0, 3 * page, len(rows)), rows)]
        say("reserve")
        third = qbn.KVPool.like(pool) if separate else pool
        st = qbn.kv_reserve(nxt, ints(rows), ints(room), out=third)
        assert int(st) == ref.reserve(rows, room)
        same(third, ref)
        ref.moves = []
        say("compact")
        pool = qbn.KVPool.like(pool) if separate else pool
        live = qbn.kv_compact(c, third, out=pool)
        assert int(live) == ref.compact()
        same(pool, ref)
        same_payload(c, before, ref.moves)
        assert (ref.refs[:int(live)] > 0).all() and (ref.refs[int(live):] == 0).all()


@pytest.mark.parametrize("pages,seqs", [(1, 1), (63, 3), (1024, 40), (5000, 700), (70001, 1500)])
def test_reserve_many(pages, seqs):
    rng = np.random.default_rng(pages)
    ps, row = 16, 64
    table = np.full((seqs, row), -1, np.int32)
    refs = (rng.random(pages) < 0.3).astype(np.int32) * rng.integers(1, 4, pages).astype(np.int32)
    pool = qbn.KVPool(torch.from_numpy(table).to(DEV), ints(np.zeros(seqs)), ints(refs), ps)
    ref = R.RefPool(table, np.zeros(seqs, np.int32), refs, ps)
    rows = rng.permutation(seqs)
    tokens = rng.integers(0, 2 * ps * max(1, min(row // 2, pages // seqs)), seqs) // 2
    say("reserve", pages, seqs)
    st = qbn.kv_reserve(pool, ints(rows), ints(tokens))
    assert int(st) == ref.reserve(rows.tolist(), tokens.tolist())
    same(pool, ref)


def test_sizes_beyond_the_near_lookups():
    """More slots, requests, pages and entries than fit the plans' LDS, with a
    failing request at the end of one call."""
    rng = np.random.default_rng(41)
    seqs, row, ps, pages = 9001, 9, 16, 60000
    table = np.full((seqs, row), -1, np.int32)
    refs = (rng.random(pages) < 0.1).astype(np.int32)
    pool = qbn.KVPool(torch.from_numpy(table).to(DEV), ints(np.zeros(seqs)), ints(refs), ps)
    ref = R.RefPool(table, np.zeros(seqs, np.int32), refs, ps)
    rows, tokens = rng.permutation(seqs)[:3000], rng.integers(0, row * ps + 1, 3000)
    say("reserve", seqs, pages)
    st = qbn.kv_reserve(pool, ints(rows), ints(tokens))
    assert int(st) == ref.reserve(rows.tolist(), tokens.tolist()) == -1
    same(pool, ref)
    other = rng.permutation(seqs)[:2500]
    st = qbn.kv_reserve(pool, ints(list(other) + [seqs]), ints([0] * 2501))
    assert int(st) == ref.reserve(list(other) + [seqs], [0] * 2501) == 2500
    same(pool, ref)
    gone = rng.permutation(seqs)[:4000]
    after = qbn.KVPool.like(pool)
    say("free", len(gone))
    qbn.kv_free(pool, ints(gone), out=after)
    ref.release(gone.tolist())
    same(after, ref)
    c = qbn.KVCache.empty("mxfp4", 1, pages, 1, ps, 64, device=DEV)
    kids = [int(b) for b in range(seqs) if ref.lens[b] == 0][:2500]
    parents = [int(b) for b in rng.choice([b for b in range(seqs) if ref.lens[b] > 0], 2500)]
    say("fork", len(kids))
    st = qbn.kv_fork(c, after, ints(parents), ints(kids))
    assert int(st) == ref.fork(parents, kids) == -1
    same(after, ref)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (20, 5), (100, 33)])
def test_free_into_other_tables(window, sinks):
    """out = in without the pages given back, in as it was."""
    rng = np.random.default_rng(window + sinks + 1)
    c, pool, ref = make(rng, pages=60, row=20, lens=(300, 16, 3, 0, 97, 320))
    pool.table[3, 2], ref.table[3, 2] = 77, 77  # no page: gone without a count
    old = [t.clone() for t in (pool.table, pool.lens, pool.refs)]
    out = qbn.KVPool.like(pool)
    rows = [0, 1, 2, 3, 5, 5, 7, -2]
    qbn.kv_free(pool, ints(rows), window=window, sinks=sinks, out=out)
    ref.release(rows, window, sinks)
    same(out, ref)
    for x, y in zip(old, (pool.table, pool.lens, pool.refs)):
        assert torch.equal(x, y)


def test_compact_keeps_entries_that_name_free_pages():
    rng = np.random.default_rng(44)
    c, pool, ref = make(rng)
    free = [p for p in range(40) if ref.refs[p] == 0]
    pool.table[5, 0], pool.table[5, 1] = free[-1], free[0]
    ref.table[5, 0], ref.table[5, 1] = free[-1], free[0]
    before = payload(c)
    qbn.kv_compact(c, pool)
    ref.compact()
    same(pool, ref)
    same_payload(c, before, ref.moves)


@pytest.mark.parametrize("rows,tokens", [
    ([0, 7], [1, 1]),           # no such slot
    ([0, -1], [1, 1]),
    ([4, 0, 4], [1, 1, 1]),     # named twice
    ([0, 1, 2], [1, 2, -1]),    # fewer tokens
    ([0], [89]),                # the row is too short: 40 + 89 > 128
    ([3, 0], [128, 10 ** 9]),
    ([3, 5, 0, 1], [128, 100, 88, 112]),  # 31 free: 8 + 7 + 5 + 7 fit
    ([3, 5, 0, 1, 2], [128, 128, 88, 112, 125]),  # 8 + 8 + 5 + 7 + 7 do not
])
def test_reserve_refusals(rows, tokens):
    rng = np.random.default_rng(1)
    c, pool, ref = make(rng)
    say("reserve", rows, tokens)
    st = qbn.kv_reserve(pool, ints(rows), ints(tokens))
    want = ref.reserve(rows, tokens)
    assert int(st) == want
    same(pool, ref)


@pytest.mark.parametrize("parents,children", [
    ([0, 6], [3, 5]), ([0, 1], [3, 6]), ([0, 3], [3, 3]), ([1, 0], [3, 3]), ([0, 0], [3, 2]), ([3], [3]),
    ([3, 0, 2], [5, 5, 3]), ([0, 3], [3, 5]), ([], []),
])
def test_fork_refusals_and_empty_parents(parents, children):
    rng = np.random.default_rng(2)
    c, pool, ref = make(rng)
    before = payload(c)
    say("fork", parents, children)
    st = qbn.kv_fork(c, pool, ints(parents), ints(children))
    assert int(st) == ref.fork(parents, children)
    same(pool, ref)
    same_payload(c, before, ref.moves)


def test_fork_without_free_pages_and_with_a_bad_tail_changes_nothing():
    rng = np.random.default_rng(3)
    c, pool, ref = make(rng, pages=9, lens=(40, 16, 3, 0, 48, 0))  # 3 + 1 + 1 + 3 used, one free
    before = payload(c)
    st = qbn.kv_fork(c, pool, ints([0, 2]), ints([3, 5]))
    assert int(st) == ref.fork([0, 2], [3, 5]) == 1
    same(pool, ref)
    pool.table[0, 2] = ref.table[0, 2] = 9
    st = qbn.kv_fork(c, pool, ints([0]), ints([3]))
    assert int(st) == ref.fork([0], [3]) == 0
    same(pool, ref)
    same_payload(c, before, [])


@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (20, 5), (16, 16), (100, 33), (1000, 0)])
def test_free_what_slid_out_of_the_window(window, sinks):
    rng = np.random.default_rng(window + sinks)
    c, pool, ref = make(rng, pages=60, row=20, lens=(300, 16, 3, 0, 97, 320))
    rows = [0, 1, 2, 4, 5, 5, 7]
    qbn.kv_free(pool, ints(rows), window=window, sinks=sinks)
    ref.release(rows, window, sinks)
    same(pool, ref)


def test_compact_of_full_empty_and_broken_tables():
    rng = np.random.default_rng(4)
    c, pool, ref = make(rng)
    pool.table[3, 0], pool.table[3, 1] = 4000, -5  # left as they are
    ref.table[3, 0], ref.table[3, 1] = 4000, -5
    for rows in ([], [0, 1, 2, 4]):
        before, ref.moves = payload(c), []
        qbn.kv_free(pool, ints(rows))
        ref.release(rows)
        live = qbn.kv_compact(c, pool)
        assert int(live) == ref.compact()
        same(pool, ref)
        same_payload(c, before, ref.moves)
    assert int(live) == 0


def test_bookkeeping_in_a_graph():
    """A turn captured into a graph, replayed three times against the eager result."""
    rng = np.random.default_rng(5)
    c, pool, _ = make(rng, pages=100, row=12, lens=(40, 16, 3, 0, 64, 0))
    out = qbn.KVPool.like(pool)
    gone, par, kid, rows, room = ints([1]), ints([0, 4]), ints([3, 5]), ints([0, 3, 5]), ints([9, 20, 1])

    def turn():
        qbn.kv_free(pool, gone, out=out)
        a = qbn.kv_fork(c, out, par, kid)
        b = qbn.kv_reserve(out, rows, room)
        return torch.cat([a, b, qbn.kv_compact(c, out)])

    first = turn()
    torch.cuda.synchronize()
    want = [t.clone() for t in (first, out.table, out.lens, out.refs, c.k, c.v, c.k_scales, c.v_scales)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = turn()
    for rep in range(3):
        for t in (got, out.table, out.lens, out.refs):
            t.fill_(77)
        torch.cuda.synchronize()
        say("graph replay", rep)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip((got, out.table, out.lens, out.refs, c.k, c.v, c.k_scales, c.v_scales), want):
            assert torch.equal(x, y)
    del g
