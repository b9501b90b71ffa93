"""GPU: the paged attention kernels where their work is cut differently: many
rows (eight waves a workgroup), many sequences (the scans of the lengths pass
64 at a time), pieces of every length, offsets beyond 32 bits, scales of every
sign. References and bounds are those of test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
from gpu_util import DEV, say
from test_gpu_kv_attention import check, decode, fill, prefill, random_cache, vectors

pytestmark = pytest.mark.gpu


def setup(fmt, dim, ps, heads, lens, rng, spare=2):
    pages = sum(-(-n // ps) for n in lens) + spare
    table = R.torch_table(lens, ps, max(lens) // ps + 2, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, rng)
    fill(c, table, lens, rng)
    return c, table


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
def test_prefill_many_rows(fmt, dim, window, sinks):
    """From 65536 rows a key-value head's worth on, tiles of 256 rows: several
    sequences, ends inside tiles, the same bits twice."""
    rng = np.random.default_rng(dim + window)
    heads, group, ps = 4, 8, 32
    lens, news = [2300, 70, 5, 131], [2100, 70, 1, 64]
    assert sum(news) * group // 256 * heads >= 256
    c, table = setup(fmt, dim, ps, heads, lens, rng)
    q = vectors(rng, sum(news), heads * group, dim, gain=2.0)
    cu = [0] + np.cumsum(news).tolist()
    out, lse = prefill(c, q, cu, table, lens, window=window, sinks=sinks)
    check(c, out, lse, q, table, lens, news, window, sinks, rows={0, 1, 31, 32, 63, 64, 69, 1027, 2098, 2099})
    again, lse2 = prefill(c, q, cu, table, lens, window=window, sinks=sinks)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_prefill_many_rows_with_infinities_and_bad_pages():
    rng = np.random.default_rng(50)
    n, ps, dim, heads, group = 2200, 16, 64, 4, 8
    c, table = setup("bf16", dim, ps, heads, [n, 40], rng)
    news = [n, 40]
    cu = [0, n, n + 40]
    q = vectors(rng, n + 40, heads * group, dim)
    clean, lse0 = prefill(c, q, cu, table, [n, 40], window=30, sinks=2)
    odd = {1: (3, float("inf")), n - 5: (7, float("nan")), 700: (9, float("-inf")), 701: (9, float("inf"))}
    for tok, (d, x) in odd.items():
        c.v[0, int(table[0, tok // ps]), 2, tok % ps, d] = x
    out, lse = prefill(c, q, cu, table, [n, 40], window=30, sinks=2)
    assert torch.equal(lse, lse0)
    got, was = out.float().cpu().numpy(), clean.float().cpu().numpy()
    want = was.copy()
    for i in range(n):
        for tok, (d, x) in odd.items():
            if tok <= i and (tok > i - 30 or tok < 2):
                with np.errstate(invalid="ignore"):
                    want[i, 2 * group:3 * group, d] += x
    special = ~np.isfinite(want)
    assert special.any() and (np.isnan(want) == np.isnan(got)).all()
    assert (got[special & ~np.isnan(want)] == want[special & ~np.isnan(want)]).all()
    touched = np.zeros(got.shape, bool)
    touched[:n, 2 * group:3 * group, [d for d, _ in odd.values()]] = True
    assert (got[~touched] == was[~touched]).all()
    bad = table.clone()
    bad[1, 1] = -1  # the second sequence's only: its tile gives NaN, the first one's rows do not change
    out2, lse2 = prefill(c, q, cu, bad, [n, 40], window=30, sinks=2)
    assert torch.isnan(out2[n:]).all() and torch.isnan(lse2[n:]).all() and torch.equal(lse2[:n], lse[:n])


@pytest.mark.parametrize("seqs", [64, 65, 200])
def test_many_sequences(seqs):
    """More sequences than a wave has lanes, empty ones among them."""
    rng = np.random.default_rng(seqs)
    ps, dim, heads, group = 16, 64, 1, 2
    lens = [int(x) for x in rng.integers(0, 400, seqs)]
    lens[0], lens[seqs // 2], lens[-1] = 0, 3000, 1
    news = [int(rng.integers(0, min(n, 4) + 1)) for n in lens]
    c, table = setup("mxfp8", dim, ps, heads, lens, rng)
    q = vectors(rng, seqs, heads * group, dim, gain=2.0)
    out, lse = decode(c, q, table, lens)
    check(c, out, lse, q, table, lens, [1] * seqs, 0, 0)
    cu = [0] + np.cumsum(news).tolist()
    q = vectors(rng, cu[-1], heads * group, dim, gain=2.0)
    out, lse = prefill(c, q, cu, table, lens)
    check(c, out, lse, q, table, lens, news, 0, 0)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_decode_pieces_of_every_length(fmt, dim):
    """One to many units of 128 tokens a piece, ends inside a unit and on its border."""
    rng = np.random.default_rng(dim)
    lens, ps = [127, 128, 384, 385, 640, 1025, 5000], 64
    c, table = setup(fmt, dim, ps, 2, lens, rng)
    wide = torch.cat([table, torch.full((len(lens), 4000), -1, dtype=torch.int32)], 1)
    q = vectors(rng, len(lens), 6, dim, gain=2.0)
    out, lse = decode(c, q, wide, lens)
    check(c, out, lse, q, table, lens, [1] * len(lens), 0, 0)
    out, lse = decode(c, q, wide, lens, window=300, sinks=9)
    check(c, out, lse, q, table, lens, [1] * len(lens), 300, 9)


@pytest.mark.parametrize("scale", [0.0, -0.0, 0.7, -1.3, 1e-30])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_scales(fmt, scale):
    rng = np.random.default_rng(7)
    lens, news, ps, dim = [300, 77], [70, 77], 32, 64
    c, table = setup(fmt, dim, ps, 1, lens, rng)
    q = vectors(rng, 147, 3, dim)
    s = float(np.float32(scale))
    out, lse = prefill(c, q, [0, 70, 147], table, lens, scale=scale, window=100, sinks=3)
    check(c, out, lse, q, table, lens, news, 100, 3, scale=s)
    out, lse = decode(c, q[:2], table, lens, scale=scale)
    check(c, out, lse, q[:2], table, lens, [1, 1], 0, 0, scale=s)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ragged", [True, False])
def test_append_many_tokens(fmt, dtype, ragged):
    """Several tokens a wave: groups of tokens that cross sequences and pages, empty
    sequences, tokens without a page, before position 0, beyond the row and beyond
    cu. Whatever is not a token's place keeps its bytes."""
    rng = np.random.default_rng(90 + ragged)
    heads, dim, ps, row = 61, 96, 16, 12
    if ragged:
        news = [1, 0, 2, 131, 0, 0, 1, 1, 61, 70, 5, 96, 3]
        lens = [n + int(rng.integers(0, 40)) for n in news]
        lens[8] = 23            # 38 of its 61 tokens stand before position 0
        lens[9] = ps * row + 9  # the last 9 stand beyond the row
        cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        tokens = int(cu[-1]) + 6  # the last 6 belong to no sequence
    else:
        tokens = 413
        news, cu = [1] * tokens, None
        lens = [int(n) for n in rng.integers(0, 2 * ps + 1, tokens)]
    table = R.torch_table([min(n, ps * row) for n in lens], ps, row, sum(-(-n // ps) for n in lens) + 3, rng)
    pages = sum(-(-n // ps) for n in lens) + 3
    table[3, 2], table[11 if ragged else 40, 0] = -1, pages
    c = random_cache(fmt, pages, heads, ps, dim, None, junk=0x5A)
    want = [t.cpu() if t is not None else None for t in (c.k, c.v, c.k_scales, c.v_scales)]
    wide = vectors(rng, tokens, 2 * heads, dim, dtype=torch.float32).to(dtype)
    dw = wide.to(DEV)
    say("append many", fmt, dtype, ragged)
    qbn.kv_append(c, dw[:, :heads], dw[:, heads:], table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                  None if cu is None else torch.from_numpy(cu).to(DEV))
    torch.cuda.synchronize()
    for which, x in ((0, wide[:, :heads]), (1, wide[:, heads:])):
        code, scale = (None, None) if fmt == "bf16" else R.quantize(fmt, x.double().numpy())
        if fmt == "mxfp4":
            code = code[..., 0::2] | (code[..., 1::2] << 4)
        t = 0
        for b, n in enumerate(news):
            for pos in range(lens[b] - n, lens[b]):
                page = int(table[b, pos // ps]) if 0 <= pos < ps * row else -1
                if 0 <= page < pages:
                    want[which][0, page, :, pos % ps] = x[t].to(torch.bfloat16) if code is None else torch.from_numpy(code[t])
                    if code is not None:
                        want[which + 2][0, page, :, :, pos % ps] = torch.from_numpy(scale[t])
                t += 1
    for got, w, name in zip((c.k, c.v, c.k_scales, c.v_scales), want, ("k", "v", "k_scales", "v_scales")):
        if w is not None:
            assert torch.equal(got.cpu().view(torch.uint8), w.view(torch.uint8)), name


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_pages_beyond_32_bit_offsets(fmt):
    """The same tokens in the first and in the last pages of a cache whose K has
    more than 2^32 bytes (bf16) or elements (4 bits) give the same bits."""
    rng = np.random.default_rng(60)
    heads, ps, dim, group, n = 8, 64, 128, 4, 700
    pages = (1 << 32) // (heads * ps * dim * 2) + 40 if fmt == "bf16" else (1 << 32) // (heads * ps * dim) + 40
    c = qbn.KVCache.empty(fmt, 1, pages, heads, ps, dim, device=DEV)
    used = -(-n // ps)
    low = torch.arange(used, dtype=torch.int32).reshape(1, -1)
    high = pages - 1 - low
    k, v = vectors(rng, n, heads, dim).to(DEV), vectors(rng, n, heads, dim).to(DEV)
    lens, cu = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)
    got = []
    for table in (low, high):
        say("append", fmt, pages)
        qbn.kv_append(c, k, v, table.to(DEV), lens, cu)
        q = vectors(np.random.default_rng(61), 90, heads * group, dim, gain=2.0)
        got.append(decode(c, q[:1], table, [n]) + prefill(c, q, [0, 90], table, [n]))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    moved = qbn.KVPool(high.to(DEV).contiguous(), lens.clone(), torch.zeros(pages, dtype=torch.int32, device=DEV), ps)
    moved.refs[high.long().to(DEV).reshape(-1)] = 1
    if pages <= 1 << 20:
        live = qbn.kv_compact(c, moved)
        torch.cuda.synchronize()
        assert int(live) == used and sorted(moved.table[0].tolist()) == list(range(used))
        out, lse = decode(c, q[:1], moved.table.cpu(), [n])
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    del c


def test_side_stream_and_given_buffers():
    """out, lse and workspace given; inputs made on another stream, which the caller orders."""
    rng = np.random.default_rng(62)
    lens, ps, dim = [3000, 20], 64, 128
    c, table = setup("mxfp8", dim, ps, 2, lens, rng)
    q = vectors(rng, 2, 8, dim).to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    t = table.to(DEV)
    want, lse0 = qbn.kv_attention_decode(c, q, t, n)
    out, lse = torch.empty_like(want), torch.empty_like(lse0)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = qbn.kv_attention_decode(c, q, t, n, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert a is out and b is lse and torch.equal(out, want) and torch.equal(lse, lse0)


def test_decode_calls_on_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own, give the bits of calls alone."""
    rng = np.random.default_rng(71)
    lens, ps, dim = [6000, 4000, 300], 64, 64
    c, table = setup("mxfp4", dim, ps, 2, lens, rng)
    t, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = [vectors(rng, 3, 8, dim).to(DEV) for _ in range(2)]
    want = [qbn.kv_attention_decode(c, q, t, n) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for rep in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(qbn.kv_attention_decode(c, qs[i], t, n))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_split_decode_in_a_graph_beside_eager_calls():
    rng = np.random.default_rng(72)
    lens, ps, dim = [6000, 900], 64, 128
    c, table = setup("mxfp8", dim, ps, 2, lens, rng)
    t, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = vectors(rng, 2, 8, dim).to(DEV)
    qbn.kv_attention_decode(c, q, t, n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = qbn.kv_attention_decode(c, q, t, n)
    for rep in range(4):
        q.copy_(vectors(rng, 2, 8, dim))
        want = qbn.kv_attention_decode(c, q, t, n)
        torch.cuda.synchronize()
        say("graph replay", rep)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    del g
