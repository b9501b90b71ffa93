"""GPU: examples/moe_decode.py (4-bit projections, append with the rotation,
prefill, decode, the choice of experts and their layer together): every stage of
every pass against binary64, from what went into it."""
import os
import sys

import numpy as np
import pytest
import torch

import kv_ref as R
import step_ref as S
from gpu_util import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_decode as E  # noqa: E402

pytestmark = pytest.mark.gpu


def numbers(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("fmt,experts_fmt", [("bf16", "mxfp4"), ("mxfp8", "nvfp4"), ("mxfp4", "mxfp4")])
def test_example_matches_binary64_stage_by_stage(fmt, experts_fmt):
    prompts = (37, 5, 64)
    seen = []
    steps = list(E.serve(fmt, experts_fmt, 5, prompts, watch=lambda *a: seen.append(
        a[:2] + tuple(t.detach().clone() for t in a[2:]))))
    assert len(seen) == 2 * E.LAYERS * len(steps) and all(int(ok) == -1 for *_, ok in steps)
    d = steps[0][1]
    f, factor = d.rope.frequencies, float(np.float32(d.rope.factor))
    # the cache after the last pass still holds every token as it was stored
    scales = (None, None) if fmt == "bf16" else (d.cache.k_scales.cpu(), d.cache.v_scales.cpu())
    held = [[R.decode(fmt, t[i].cpu(), None if s is None else s[i]) for t, s in zip((d.cache.k, d.cache.v), scales)]
            for i in range(E.LAYERS)]
    table = d.pool.table.cpu().numpy()
    layers = [[S.decode(experts_fmt, w.cpu().numpy(), s.cpu().numpy(), None if f2 is None else f2.cpu().numpy())
               for w, s, f2 in ((m.w13, m.w13_scales, m.w13_scale2), (m.w2, m.w2_scales, m.w2_scale2))] for m in d.moe]
    lens = np.zeros(len(prompts), int)
    for n, (what, _, _, _, _) in enumerate(steps):
        news = list(prompts) if what == "prefill" else [1] * len(prompts)
        lens = lens + news
        pos = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, news)])
        for i in range(E.LAYERS):
            say(fmt, experts_fmt, what, n, "layer", i)
            kind, layer, v, turned, a = seen[(n * E.LAYERS + i) * 2]
            assert (kind, layer) == ("attention", i)
            v, turned, a = numbers(v), numbers(turned), numbers(a)
            want, tol = S.turn(v[:, :E.HEADS], pos, f, "half", factor)
            assert (np.abs(turned - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
            # what the cache holds of these tokens
            kk, tol = S.turn(v[:, E.HEADS:E.HEADS + E.KV], pos, f, "half", factor)
            where = [(b, p) for b, (m, t) in enumerate(zip(lens, news)) for p in range(m - t, m)]
            page = np.array([table[b, p // E.PAGE] for b, p in where])
            slot = np.array([p % E.PAGE for _, p in where])
            for part, y, t in ((0, kk, tol), (1, v[:, E.HEADS + E.KV:], 0.0)):
                if fmt == "bf16":
                    assert (np.abs(held[i][part][page, :, slot] - y) <= t + 2.0 ** -8 * (np.abs(y) + t)).all()
                else:
                    codes = (d.cache.k, d.cache.v)[part][i].cpu().numpy()[page, :, slot]
                    S.check_block(fmt, codes, scales[part][i].numpy()[page, :, :, slot], y, t + np.zeros_like(y), "cache")
            at = 0
            for b, (m, t) in enumerate(zip(lens, news)):
                for h in range(E.HEADS):
                    rows = [R.rows_of(held[i][p], table[b], m, h // (E.HEADS // E.KV)) for p in (0, 1)]
                    for j in range(t):
                        o, l, w, reach, count = R.attention(turned[at + j, h], *rows, m - t + j, 0, 0, E.DIM ** -0.5)
                        to, _ = R.attention_tolerance(E.DIM, o, w, l, reach, count)
                        assert (np.abs(a[at + j, h] - o) <= to).all()
                at += t
            kind, layer, x, y, ids, weights = seen[(n * E.LAYERS + i) * 2 + 1]
            assert (kind, layer) == ("experts", i)
            x, y, ids, weights = numbers(x), numbers(y), ids.cpu().numpy(), numbers(weights)
            want, share, gap = S.route(x, numbers(d.moe[i].router.weight), None, E.TOP, True)
            assert gap > 1e-12 and np.array_equal(ids, want)
            assert (np.abs(weights - share) <= share * 2.0 ** -24 * 1.001).all()
            want, tol = S.experts(x, ids, weights, *layers[i])
            assert (np.abs(y - want) <= tol).all()
