"""GPU: the paged attention kernels at the ends of the formats: every scale byte
with every code, scores far from zero and infinite ones, infinities and NaN of
V in tokens that only some rows see."""
import math

import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
from gpu_util import DEV
from test_gpu_kv_attention import decode, fill, prefill, random_cache, vectors

pytestmark = pytest.mark.gpu

INF = float("inf")


def one_token_each(fmt, part):
    """A cache of 256 pages, page b with one token whose scale bytes of K or V are
    all b, its elements every code in turn; head_dim 256. The table and lengths of
    a sequence each, and the values that the codes stand for."""
    c = qbn.KVCache.empty(fmt, 1, 256, 1, 16, 256, device=DEV)
    c.k.zero_(), c.v.zero_(), c.k_scales.fill_(127), c.v_scales.fill_(127)
    if fmt == "mxfp8":
        codes = torch.arange(256, dtype=torch.uint8)
        if part == "k":
            codes[[127, 255]] = 0  # NaN times the query's zeros would be everywhere
    else:
        codes = torch.tensor([2 * i % 16 | (2 * i + 1) % 16 << 4 for i in range(128)], dtype=torch.uint8)
    x, s = (c.k, c.k_scales) if part == "k" else (c.v, c.v_scales)
    x[0, :, 0, 0] = codes.to(DEV)
    s[0, :, 0, :, 0] = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None]
    with np.errstate(all="ignore"):
        values = R.decode(fmt, x[0].cpu(), s[0].cpu())[:, 0, 0]
    return c, torch.arange(256, dtype=torch.int32).reshape(-1, 1), [1] * 256, torch.from_numpy(values)


def calls(c, q, table, lens):
    yield decode(c, q, table, lens)
    yield prefill(c, q, list(range(len(lens) + 1)), table, lens)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_every_scale_byte_with_every_code_of_v(fmt):
    """A sequence of one token returns it: the value rounded to bfloat16 (which
    all but those below 2^-133 and beyond the largest fit), NaN for byte 255."""
    c, table, lens, v = one_token_each(fmt, "v")
    want = v.float().bfloat16()  # binary32 holds them all but the overflowing ones
    q = torch.zeros(256, 1, 256, dtype=torch.bfloat16)
    for out, lse in calls(c, q, table, lens):
        got = out[:, 0].cpu()
        assert (torch.isnan(got) == torch.isnan(want)).all()
        ok = torch.isnan(want) | (got == want)
        assert ok.all(), "scale bytes %s" % sorted(set((~ok).nonzero()[:, 0].tolist()))
        assert torch.isnan(want[255]).all() and (lse == 0).all()


@pytest.mark.parametrize("fmt,top", [("mxfp8", 246), ("mxfp4", 252)])
def test_every_scale_byte_with_every_code_of_k(fmt, top):
    """256 query heads, head h with a 1 at element h: lse is that element's score.
    Bytes up to the largest whose products fit bfloat16, and 255, which is NaN."""
    c, table, lens, k = one_token_each(fmt, "k")
    q = torch.eye(256, dtype=torch.bfloat16).expand(256, 256, 256)
    scale = 1 / 16
    for out, lse in calls(c, q, table, lens):
        got, want = lse.double().cpu()[:top + 1], k[:top + 1].float().bfloat16().double() * scale
        # the factor scale log2 e, its product, the product with log 2: three roundings and the constants'; below 2^-126 maybe 0
        err = (got - want).abs()
        assert (err <= 6 * 2.0 ** -24 * want.abs() + 2.0 ** -125).all()
        assert torch.isnan(lse[255]).all() and torch.isnan(out[255]).all()
        assert (out[:top + 1] == 0).all()


@pytest.mark.parametrize("size", [1e6, 3e8, 1e10, 1e13, 1e20, 1e36])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("wide", [False, True])
def test_scores_far_from_zero(size, sign, wide):
    """Scores of a few values, so far apart that only the largest has a weight: the
    mean of V over its tokens. They differ by 2^-6 of themselves, more than 10^4,
    and binary32 holds them to 2^-22, below a hundredth where they are small."""
    rng = np.random.default_rng(9)
    n, t, ps, dim = 1700, 5, 32, 64
    table = R.torch_table([n], ps, 54, 54, rng)
    c = random_cache("bf16", 54, 1, ps, dim, rng)
    _, v = fill(c, table, [n], rng)
    level = torch.from_numpy(rng.integers(0, 3, n))
    level[-t - 40:] = 1  # the last rows see the same largest
    score = (sign * size * (1 - level.double() / 64)).to(torch.bfloat16)
    for j in range(n):
        c.k[0, int(table[0, j // ps]), 0, j % ps] = 0
        c.k[0, int(table[0, j // ps]), 0, j % ps, 7] = score[j]
    if wide:
        table = torch.cat([table, torch.full((1, 400), -1, dtype=torch.int32)], 1)
    q = torch.zeros(t, 2, dim, dtype=torch.bfloat16)
    q[:, :, 7] = 1
    top = score.double().max()
    on = score.double() == top
    want, weight = v[on, 0].double().mean(0).numpy(), v[on, 0].double().abs().mean(0).numpy()
    lse0 = float(top) + math.log(int(on.sum()))
    for out, lse in (decode(c, q[:1], table, [n], scale=1.0), prefill(c, q, [0, t], table, [n], scale=1.0)):
        err = np.abs(out.double().cpu().numpy() - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + n * 2.0 ** -23) * weight).all()
        assert ((lse.double().cpu() - lse0).abs() <= 6 * 2.0 ** -24 * abs(lse0)).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("how", ["infinite", "overflow"])
def test_scores_of_minus_infinity(fmt, wide, how):
    """Where every visible score is -inf, out is 0 and lse -inf; where only some
    are, those tokens do not count; a score of +inf gives NaN."""
    if how == "overflow" and fmt != "bf16":
        pytest.skip("the MX formats reach infinity in their expansion")
    rng = np.random.default_rng(3)
    n, ps, dim = 700, 16, 64
    table = R.torch_table([n], ps, 45, 45, rng)
    c = random_cache(fmt, 45, 1, ps, dim, rng)
    fill(c, table, [n], rng)
    clean_k, clean_s = c.k.clone(), None if fmt == "bf16" else c.k_scales.clone()
    if wide:
        table = torch.cat([table, torch.full((1, 400), -1, dtype=torch.int32)], 1)
    q = vectors(rng, 3, 2, dim)
    q[..., :32] = q[..., :32].abs() * (1e30 if how == "overflow" else 1)
    if how == "overflow":
        q[..., 32:] = 0
    big = 3e38 if how == "overflow" else INF

    def put(tokens, sign):  # K's first elements so large that the score is infinite
        for t in tokens:
            p, i = int(table[0, t // ps]), t % ps
            if fmt == "bf16":
                c.k[0, p, 0, i, :32 if how == "overflow" else 1] = sign * big
            else:
                c.k_scales[0, p, 0, 0, i] = 254
                code = {"mxfp8": 0x7E, "mxfp4": 0x77}[fmt] | (0 if sign > 0 else {"mxfp8": 0x80, "mxfp4": 0x88}[fmt])
                c.k[0, p, 0, i, :32 if fmt == "mxfp8" else 16] = code

    put(range(n), -1)
    for out, lse in (decode(c, q[:1], table, [n]), prefill(c, q, [0, 3], table, [n])):
        assert (out == 0).all() and (lse == -INF).all()
    c.k.copy_(clean_k)
    if clean_s is not None:
        c.k_scales.copy_(clean_s)
    some = [0, 5, 64, 127, 128, 300, n - 3]
    put(some, -1)
    scale = 1e-30 if how == "overflow" else dim ** -0.5
    with np.errstate(all="ignore"):
        k = R.decode(fmt, c.k[0].cpu(), None if fmt == "bf16" else c.k_scales[0].cpu())
        v = R.decode(fmt, c.v[0].cpu(), None if fmt == "bf16" else c.v_scales[0].cpu())
    kk, vv = R.rows_of(k, table[0].tolist(), n, 0), R.rows_of(v, table[0].tolist(), n, 0)
    keep = np.setdiff1d(np.arange(n), some)
    for out, lse, first in (decode(c, q[:1], table, [n], scale=scale) + (n - 1,),
                            prefill(c, q, [0, 3], table, [n], scale=scale) + (n - 3,)):
        for i in range(out.shape[0]):
            on = keep[keep <= first + i]
            for h in range(2):
                o, l, w, reach, count = R.attention(q[i, h].double().numpy(), kk[on], vv[on], len(on) - 1, 0, 0, float(np.float32(scale)))
                to, tl = R.attention_tolerance(dim, o, w, l, reach, count)
                assert (np.abs(out[i, h].double().cpu().numpy() - o) <= to).all() and abs(float(lse[i, h]) - l) <= tl
    if how == "infinite":
        put([9], 1)
        for out, lse in (decode(c, q[:1], table, [n]), prefill(c, q, [0, 3], table, [n])):
            assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("few", [True, False])
def test_prefill_infinities_in_masked_tokens_of_the_mx_formats(fmt, few):
    """An infinity or NaN of V, here of a block of 32, reaches exactly the rows that
    see its token; rows that see none keep their bits."""
    rng = np.random.default_rng(23)
    n, ps, dim, window, sinks = 1600, 16, 96, 30, 2
    t = 20 if few else 1600  # few rows: the split form
    table = R.torch_table([n], ps, 100, 100, rng)
    c = random_cache(fmt, 100, 1, ps, dim, rng)
    fill(c, table, [n], rng)
    q = vectors(rng, t, 1, dim)
    clean, lse0 = prefill(c, q, [0, t], table, [n], window=window, sinks=sinks)
    wide = 32 if fmt == "mxfp8" else 16
    codes = {"mxfp8": (0x7E, 0xFE), "mxfp4": (0x77, 0xFF)}[fmt]
    odd = {0: (0, INF), 1: (0, -INF), n - 5: (1, math.nan), n - 12: (2, -INF), n - 300: (2, INF), n - 290: (1, math.nan)}
    for tok, (blk, x) in odd.items():
        p, i = int(table[0, tok // ps]), tok % ps
        if math.isnan(x) and fmt == "mxfp8" and tok == n - 5:
            c.v[0, p, 0, i, blk * wide:(blk + 1) * wide] = 0x7F  # the code
        elif math.isnan(x):
            c.v_scales[0, p, 0, blk, i] = 255
        else:
            c.v_scales[0, p, 0, blk, i] = 254
            c.v[0, p, 0, i, blk * wide:(blk + 1) * wide] = codes[x < 0]
    out, lse = prefill(c, q, [0, t], table, [n], window=window, sinks=sinks)
    assert torch.equal(lse, lse0)
    got, was = out[:, 0].float().cpu().numpy(), clean[:, 0].float().cpu().numpy()
    want, sees = was.copy(), np.zeros(t, bool)
    for i in range(t):
        pos = n - t + i
        for tok, (blk, x) in odd.items():
            if tok <= pos and (tok > pos - window or tok < sinks):
                sees[i] = True
                with np.errstate(invalid="ignore"):
                    want[i, 32 * blk:32 * blk + 32] += x
    special = ~np.isfinite(want)
    assert special.any() and (np.isnan(want) == np.isnan(got)).all()
    assert (got[special & ~np.isnan(want)] == want[special & ~np.isnan(want)]).all()
    assert (got[~sees] == was[~sees]).all()
    assert few or (~sees).sum() == 0 or sees.sum() > 0
