"""GPU: the choice of experts and the experts' layer against binary64."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import step_ref as S
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

FORMATS = ["mxfp4", "nvfp4"]


def router(w, top, bias=None, normalize=True):
    return qbn.MoERouter(w.to(DEV), top, None if bias is None else torch.from_numpy(bias).to(DEV), normalize)


def to(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


def make(parts, fmt, r=None):
    c13, s13, f13, c2, s2, f2 = parts
    return qbn.MoE(fmt, r, to(c13), to(s13), to(c2), to(s2), to(f13), to(f2))


def check_route(got, x, w, bias, top, normalize):
    ids, weights = got
    want, share, gap = S.route(x.double().numpy(), w.double().numpy(), None if bias is None else bias.astype(np.float64),
                               top, normalize)
    assert gap > 1e-12  # the inputs leave no doubt in binary64
    assert np.array_equal(ids.cpu().numpy(), want)
    # binary64 softmax, rounded once
    assert (np.abs(weights.cpu().double().numpy() - share) <= share * 2.0 ** -24 * 1.001 + 1e-45).all()


@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 16, 17, 100])
@pytest.mark.parametrize("experts,top,hidden", [(1, 1, 32), (2, 1, 96), (8, 2, 160), (64, 6, 1024), (128, 8, 2080), (65, 32, 64),
                                                (300, 9, 64), (1000, 17, 32), (1024, 32, 32)])
@pytest.mark.parametrize("normalize,biased", [(True, False), (False, True)])
def test_route(tokens, experts, top, hidden, normalize, biased):
    rng = np.random.default_rng(tokens * 1000 + experts)
    x, w = S.bf16(rng, tokens, hidden), S.bf16(rng, experts, hidden, gain=2 * hidden ** -0.5)
    bias = rng.standard_normal(experts).astype(np.float32) if biased else None
    say("route", tokens, experts, top, hidden)
    check_route(qbn.moe_route(router(w, top, bias, normalize), x.to(DEV)), x, w, bias, top, normalize)


def test_route_many_tokens():
    """Beyond a portion of the workspace, rows inside a wider matrix."""
    rng = np.random.default_rng(1)
    x, w = S.bf16(rng, 4100, 64), S.bf16(rng, 20, 64, gain=0.3)
    wide = torch.zeros(4100, 96, dtype=torch.bfloat16, device=DEV)
    wide[:, 16:80] = x.to(DEV)
    say("route many")
    check_route(qbn.moe_route(router(w, 3), wide[:, 16:80]), x, w, None, 3, True)


@pytest.mark.parametrize("tokens", [2, 40])
def test_route_ties_go_to_the_lowest_number(tokens):
    w = torch.zeros(130, 32, dtype=torch.bfloat16)
    w[7], w[70], w[129] = 1, 1, 1
    x = torch.ones(tokens, 32, dtype=torch.bfloat16)
    say("ties")
    ids, weights = qbn.moe_route(router(w, 6), x.to(DEV))
    assert ids.tolist() == [[7, 70, 129, 0, 1, 2]] * tokens
    assert torch.equal(weights[:, 0], weights[:, 2]) and torch.equal(weights[:, 3], weights[:, 5])
    ids, _ = qbn.moe_route(router(w, 3, bias=np.full(130, -0.0, np.float32)), -x.to(DEV))  # 0 and -0 are equal
    assert ids.tolist() == [[0, 1, 2]] * tokens


@pytest.mark.parametrize("tokens", [3, 20])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_without_a_softmax(tokens, normalize):
    """A logit of NaN or +inf, or none above -inf: NaN weights, valid experts; the
    other tokens as ever. Masked experts (-inf, the lowest value) are never chosen
    before others."""
    rng = np.random.default_rng(2)
    x, w = S.bf16(rng, tokens, 64), S.bf16(rng, 70, 64, gain=0.3)
    bias = np.zeros(70, np.float32)
    bias[3], bias[69] = -np.inf, np.finfo(np.float32).min
    x[1, 5] = float("nan")
    x[2, 6] = float("inf")
    say("no softmax")
    ids, weights = qbn.moe_route(router(w, 5, bias, normalize), x.to(DEV))
    ids, weights = ids.cpu().numpy(), weights.cpu().numpy()
    for t in range(tokens):
        assert len(set(ids[t])) == 5 and ids[t].min() >= 0 and ids[t].max() < 70
    assert np.isnan(weights[1:3]).all() and np.isfinite(weights[0]).all() and np.isfinite(weights[3:]).all()
    assert not np.isin(ids[[0] + list(range(3, tokens))], (3, 69)).any()
    masked = np.full(70, -np.inf, np.float32)
    ids, weights = qbn.moe_route(router(w, 2, masked, normalize), x[:1].to(DEV))
    assert ids.tolist() == [[0, 1]] and torch.isnan(weights).all()
    masked[11] = 0.0
    ids, weights = qbn.moe_route(router(w, 2, masked, normalize), x[:1].to(DEV))
    assert ids.tolist() == [[11, 0]] and weights.tolist() == [[1.0, 0.0]]


def test_route_large_values_stay_finite():
    """Logits beyond binary32: the sums are binary64."""
    x = torch.full((2, 32), 1e20, dtype=torch.bfloat16)
    w = torch.zeros(4, 32, dtype=torch.bfloat16)
    w[2], w[1] = 1e20, -1e20
    ids, weights = qbn.moe_route(router(w, 2, normalize=False), x.to(DEV))
    assert ids.tolist() == [[2, 0]] * 2 and weights.tolist() == [[1.0, 0.0]] * 2


def check_experts(got, x, ids, weights, parts, fmt):
    c13, s13, f13, c2, s2, f2 = parts
    want, tol = S.experts(x.double().numpy(), ids, weights.astype(np.float64), S.decode(fmt, c13, s13, f13),
                          S.decode(fmt, c2, s2, f2))
    g = got.cpu().double().numpy()
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), "%d of %d outputs off, first at %s: %r for %r +- %g" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], want[bad][0], tol[bad][0])


def choice(rng, tokens, experts, top):
    ids = np.stack([rng.permutation(experts)[:top] for _ in range(tokens)]).astype(np.int32)
    return ids, rng.uniform(0.1, 1.0, (tokens, top)).astype(np.float32)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,experts,top", [(1, 1, 1), (1, 8, 2), (1, 64, 8), (2, 4, 3), (7, 5, 2), (16, 3, 2), (33, 2, 1),
                                                (64, 1, 1), (32, 4, 2), (65, 2, 1), (40, 6, 3), (130, 3, 2), (20, 40, 5)])
@pytest.mark.parametrize("hidden,inter", [(32, 32), (96, 160), (256, 128), (160, 288)])
def test_experts(fmt, tokens, experts, top, hidden, inter):
    rng = np.random.default_rng(tokens * 100 + hidden)
    parts = S.layer(rng, fmt, experts, hidden, inter)
    x = S.bf16(rng, tokens, hidden)
    ids, weights = choice(rng, tokens, experts, top)
    say("experts", fmt, tokens, experts, top, hidden, inter)
    got = qbn.moe_experts(make(parts, fmt), x.to(DEV), to(ids), to(weights))
    check_experts(got, x, ids, weights, parts, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [1, 9, 64, 100])
def test_experts_long_rows(fmt, tokens):
    rng = np.random.default_rng(tokens)
    parts = S.layer(rng, fmt, 4, 1056, 544)
    x = S.bf16(rng, tokens, 1056)
    ids, weights = choice(rng, tokens, 4, 2)
    say("experts long", fmt, tokens)
    check_experts(qbn.moe_experts(make(parts, fmt), x.to(DEV), to(ids), to(weights)), x, ids, weights, parts, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,top", [(3, 4), (30, 6)])
def test_ids_that_are_none_and_twice(fmt, tokens, top):
    """Ids outside the experts add nothing, whatever their weight; the same expert
    twice counts twice; a token without experts gives 0."""
    rng = np.random.default_rng(8)
    parts = S.layer(rng, fmt, 3, 64, 32)
    x = S.bf16(rng, tokens, 64)
    ids, weights = rng.integers(0, 3, (tokens, top)).astype(np.int32), rng.uniform(0.1, 1, (tokens, top)).astype(np.float32)
    ids[0] = [-1, 3, 2**31 - 1, -2**31] + [7] * (top - 4)
    ids[1, 1], weights[1, 1] = -5, np.nan
    weights[0] = np.inf
    ids[2] = 1
    say("none and twice", fmt, tokens)
    got = qbn.moe_experts(make(parts, fmt), x.to(DEV), to(ids), to(weights))
    assert (got[0] == 0).all()
    check_experts(got, x, ids, np.where((ids < 0) | (ids > 2), 0, weights), parts, fmt)
    ids[:] = -1
    assert (qbn.moe_experts(make(parts, fmt), x.to(DEV), to(ids), to(weights)) == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [5, 90])
def test_bad_values_stay_with_their_token_and_expert(fmt, tokens):
    """NaN and infinities of one token reach that token alone, NaN scales of one
    expert the tokens that chose it; also in the last, partial step along k."""
    rng = np.random.default_rng(tokens)
    parts = S.layer(rng, fmt, 4, 96, 160)
    x = S.bf16(rng, tokens, 96)
    ids, weights = choice(rng, tokens, 3, 2)  # expert 3 only where set below
    ids[4] = [3, 0]
    x[2, 95], x[3, 0] = float("nan"), float("inf")
    parts[1][3, :, -1] = 255 if fmt == "mxfp4" else 0x7F
    say("bad values", fmt, tokens)
    got = qbn.moe_experts(make(parts, fmt), x.to(DEV), to(ids), to(weights)).cpu()
    assert torch.isnan(got[2]).all() and torch.isnan(got[4]).all() and not torch.isfinite(got[3]).any()
    rest = [t for t in range(tokens) if t not in (2, 3, 4)]
    parts[1][3] = 0 if fmt == "mxfp4" else 0x38
    check_experts(got[rest], x[rest], ids[rest], weights[rest], parts, fmt)


@pytest.mark.parametrize("tokens", [1, 70])
def test_every_scale_byte_and_code(tokens):
    """MXFP4 blocks of every code under every scale byte that keeps the sums finite."""
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (16, 1, 1)).reshape(1, 256, 16)  # rows of 32
    for lo in range(40, 200, 32):
        s13 = (lo + np.arange(256) % 32).astype(np.uint8).reshape(1, 256, 1)
        s13[0, 128:] = 254 - s13[0, :128]  # the up projection's undo the gate's
        c2 = np.full((1, 32, 64), 0x22, np.uint8)
        parts = [codes, s13, None, c2, np.full((1, 32, 4), 127, np.uint8), None]
        x = S.bf16(np.random.default_rng(lo), tokens, 32)
        ids, weights = np.zeros((tokens, 1), np.int32), np.ones((tokens, 1), np.float32)
        say("scale bytes", lo)
        got = qbn.moe_experts(make(parts, "mxfp4"), x.to(DEV), to(ids), to(weights))
        check_experts(got, x, ids, weights, parts, "mxfp4")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [1, 6, 50, 300])
def test_layer_is_its_two_halves(fmt, tokens):
    rng = np.random.default_rng(tokens)
    parts = S.layer(rng, fmt, 12, 128, 64)
    x, w = S.bf16(rng, tokens, 128), S.bf16(rng, 12, 128, gain=0.2)
    layer = make(parts, fmt, router(w, 3, rng.standard_normal(12).astype(np.float32), False))
    xd = x.to(DEV)
    say("layer", fmt, tokens)
    out, ids, weights = qbn.moe(layer, xd)
    ids2, weights2 = qbn.moe_route(layer.router, xd)
    assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
    assert torch.equal(out, qbn.moe_experts(layer, xd, ids, weights))
    assert torch.equal(out, qbn.moe(layer, xd)[0])  # the same bits again
    check_experts(out, x, ids.cpu().numpy(), weights.cpu().numpy(), parts, fmt)


def test_given_outputs_and_workspaces():
    """Rows inside wider matrices, given outputs, a workspace of any content that
    calls of different sizes share."""
    rng = np.random.default_rng(4)
    parts = S.layer(rng, "mxfp4", 6, 96, 64)
    w = S.bf16(rng, 6, 96, gain=0.3)
    layer = make(parts, "mxfp4", router(w, 2))
    ws = torch.full((qbn.moe_nbytes(layer.router, layer, 100, 2),), 0xFF, dtype=torch.uint8, device=DEV)
    for tokens in (100, 3, 40):
        wide = torch.full((tokens, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        x = S.bf16(rng, tokens, 96)
        wide[:, 8:104] = x.to(DEV)
        to_wide = torch.full((tokens, 120), 9.0, dtype=torch.bfloat16, device=DEV)
        ids = torch.empty(tokens, 2, dtype=torch.int32, device=DEV)
        weights = torch.empty(tokens, 2, device=DEV)
        say("given", tokens)
        out, i, v = qbn.moe(layer, wide[:, 8:104], out=to_wide[:, 16:112], ids=ids, weights=weights, workspace=ws)
        assert out.data_ptr() == to_wide[:, 16:].data_ptr() and i is ids or i.data_ptr() == ids.data_ptr()
        assert torch.equal(out, qbn.moe(layer, x.to(DEV))[0])
        assert (to_wide[:, :16] == 9).all() and (to_wide[:, 112:] == 9).all()
    with pytest.raises(ValueError, match="workspace holds"):
        qbn.moe(layer, x.to(DEV), workspace=ws[:8])


def test_empty():
    rng = np.random.default_rng(4)
    layer = make(S.layer(rng, "mxfp4", 2, 32, 32), "mxfp4", router(S.bf16(rng, 2, 32), 2))
    out, ids, weights = qbn.moe(layer, torch.empty(0, 32, dtype=torch.bfloat16, device=DEV))
    assert out.shape == (0, 32) and ids.shape == (0, 2) and weights.shape == (0, 2)


def test_refusals():
    rng = np.random.default_rng(4)
    layer = make(S.layer(rng, "mxfp4", 4, 64, 32), "mxfp4", router(S.bf16(rng, 4, 64), 2))
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV)
    ids, weights = torch.zeros(3, 2, dtype=torch.int32, device=DEV), torch.zeros(3, 2, device=DEV)
    for bad, error in ((x.float(), TypeError), (x[:, :32], ValueError), (x.cpu(), ValueError), (x[0], ValueError),
                       (torch.zeros(64, 3, dtype=torch.bfloat16, device=DEV).t(), ValueError)):
        with pytest.raises(error):
            qbn.moe(layer, bad)
        with pytest.raises(error):
            qbn.moe_route(layer.router, bad)
        with pytest.raises(error):
            qbn.moe_experts(layer, bad, ids, weights)
    with pytest.raises(qbn.QbnError):  # out over x
        qbn.moe(layer, x, out=x)
    with pytest.raises(qbn.QbnError):  # rows that are not 16-byte pieces
        qbn.moe(layer, torch.zeros(3, 68, dtype=torch.bfloat16, device=DEV)[:, :64])
    with pytest.raises(qbn.QbnError):  # one row read three times
        qbn.moe(layer, x[:1].expand(3, -1))
    with pytest.raises(TypeError):
        qbn.moe_experts(layer, x, ids.long(), weights)
    with pytest.raises(ValueError):
        qbn.moe_experts(layer, x, ids, weights[:, :1])
    with pytest.raises(qbn.QbnError):  # top_k of 33
        qbn.moe_experts(layer, x, torch.zeros(3, 33, dtype=torch.int32, device=DEV), torch.zeros(3, 33, device=DEV))
    with pytest.raises(ValueError, match="no router"):
        qbn.moe(make(S.layer(rng, "mxfp4", 4, 64, 32), "mxfp4"), x)


@pytest.mark.parametrize("tokens", [1, 20, 80])
def test_graph_replays(tokens):
    """Captured once, replayed on new inputs, between eager calls on the same workspace."""
    rng = np.random.default_rng(tokens)
    layer = make(S.layer(rng, "mxfp4", 8, 128, 64), "mxfp4", router(S.bf16(rng, 8, 128, gain=0.2), 2))
    x = S.bf16(rng, tokens, 128).to(DEV)
    ws = torch.empty(qbn.moe_nbytes(layer.router, layer, tokens, 2), dtype=torch.uint8, device=DEV)
    out, ids, weights = qbn.moe(layer, x, workspace=ws)
    say("graph", tokens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qbn.moe(layer, x, out=out, ids=ids, weights=weights, workspace=ws)
    for _ in range(4):
        x.copy_(S.bf16(rng, tokens, 128))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want, ids2, weights2 = qbn.moe(layer, x, workspace=ws)
        assert torch.equal(got, want) and torch.equal(ids, ids2) and torch.equal(weights, weights2)
