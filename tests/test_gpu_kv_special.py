"""GPU: the paged attention kernels at the ends of the formats: every scale byte
with every code, scores far from zero."""
import math

import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
from gpu_util import DEV, say
from test_gpu_kv_attention import decode, fill, prefill, random_cache

pytestmark = pytest.mark.gpu


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
